// C ABI of the feed-forward products with an epilogue, their gradients and the
// AdamW step (declarations and argument contracts in include/paro.h).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <string>
#include <utility>
#include <vector>

#include "paro_internal.h"
#include "w4_epilogue.h"

namespace paro {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int fail(int status, const std::string& msg) {
  set_error(msg);
  return status;
}

int hip_fail(hipError_t e, const char* what) { return fail(PARO_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e)); }

size_t a256(size_t b) { return (b + 255) & ~(size_t)255; }

bool known_act(int32_t act) { return act >= PARO_ACT_NONE && act <= PARO_ACT_RELU; }

// The checks of a gated call beyond those of a product with 2 N rows: an even
// split of the rows, and 32-bit offsets from a gate row to its up row.
int check_gated(const std::string& f, int64_t N, int64_t d) {
  if (N <= 0 || N % 16) return fail(PARO_ERR_SHAPE, f + ": N must be a positive multiple of 16");
  if (N > (int64_t(1) << 29) || (d > 0 && N * d >= (int64_t(1) << 31)))
    return fail(PARO_ERR_UNSUPPORTED, f + ": N * d must be below 2^31");
  return PARO_OK;
}

// One product with an epilogue, N output channels.
int run_forward(const char* fn, int epi, const paro_rotation* r, const uint16_t* x, const uint8_t* qweight,
                const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, const uint16_t* residual,
                int32_t act, uint16_t* y, int64_t M, int64_t N, int64_t d, int32_t group, void* workspace,
                size_t workspace_bytes, hipStream_t stream) {
  const std::string f(fn);
  const bool gated = epi == kEpiGated;
  if (!known_act(act)) return fail(PARO_ERR_VALUE, f + ": unknown activation");
  if (gated) {
    const int st = check_gated(f, N, d);
    if (st != PARO_OK) return st;
  }
  const int64_t P = gated ? 2 * N : N;
  bool noop = false;
  const int st = check_w4_linear(fn, r, x, qweight, scales, zeros, bias, y, M, P, d, group, &noop);
  if (st != PARO_OK || noop) return st;
  if (!aligned16(residual)) return fail(PARO_ERR_ALIGN, f + ": residual must be 16-byte aligned");
  // (X' given and few tokens: kernels without partial sums in memory)
  const size_t need = !r && M <= kDecodeMaxM ? kDecodeCounterBytes : w4_linear_min_workspace(r, M, P, d);
  if (need && (!workspace || workspace_bytes < need))
    return fail(PARO_ERR_WORKSPACE, f + ": workspace missing or smaller than the minimum");
  if ((uintptr_t)workspace & 255) return fail(PARO_ERR_ALIGN, f + ": workspace must be 256-byte aligned");
  W4Epilogue ep;
  ep.aux = residual;
  ep.act = act;
  return run_w4_product(epi, ep, r, x, qweight, scales, zeros, bias, y, M, N, d, group, (char*)workspace,
                        workspace ? workspace_bytes : 0, stream);
}

// Workspace of a backward call: the arrival counters (in every call, so that a
// workspace used for calls of several kinds keeps them zero), the recomputed
// product's partial tiles (product: whether there is one), then the input
// gradient's scratch.
size_t product_scratch(bool product, int64_t M, int64_t P, int64_t d) {
  return kDecodeCounterBytes + (product ? a256(plan_w4_gemm(M, P, d).partial_bytes) : 0);
}

int run_backward(const char* fn, bool gated, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                 const uint8_t* zeros, const uint16_t* bias, int32_t act, const uint16_t* dy, uint16_t* dz,
                 uint16_t* dx, int64_t M, int64_t N, int64_t d, int32_t group, void* workspace,
                 size_t workspace_bytes, hipStream_t stream) {
  const std::string f(fn);
  if (!known_act(act)) return fail(PARO_ERR_VALUE, f + ": unknown activation");
  if (gated) {
    const int st = check_gated(f, N, d);
    if (st != PARO_OK) return st;
  }
  const int64_t P = gated ? 2 * N : N;
  const bool product = gated || act != PARO_ACT_NONE;  // whether dz has to be computed
  if (P > (int64_t(1) << 21)) return fail(PARO_ERR_UNSUPPORTED, f + ": at most 2^21 weight rows");
  // (without a product x is not read and dz may be NULL: dy stands in for them in the checks)
  bool noop = false;
  const int st = check_w4_linear(fn, nullptr, product ? x : dy, qweight, scales, zeros, product ? bias : nullptr,
                                 product ? dz : dy, M, P, d, group, &noop);
  if (st != PARO_OK || noop) return st;
  if (!dy) return fail(PARO_ERR_NULL, f + ": NULL tensor");
  if (!aligned16(dy) || !aligned16(dz) || !aligned16(dx))
    return fail(PARO_ERR_ALIGN, f + ": dy, dz and dx must be 16-byte aligned");
  const bool copy = !product && dz && dz != dy;  // dZ = dY, for a caller who gave a place for it
  if (!product && !dx && !copy) return PARO_OK;
  const size_t first = product_scratch(product, M, P, d);
  const size_t need = first + (dx ? input_grad_scratch_bytes(M, P, d) : 0);
  if ((product || dx) && (!workspace || workspace_bytes < need))
    return fail(PARO_ERR_WORKSPACE, f + ": workspace missing or smaller than the size reported for these arguments");
  if ((uintptr_t)workspace & 255) return fail(PARO_ERR_ALIGN, f + ": workspace must be 256-byte aligned");
  char* ws = (char*)workspace;
  hipError_t e = hipSuccess;
  if (copy) {
    const size_t bytes = (size_t)M * (size_t)N * 2;  // (N % 16 == 0)
    e = launch_stream_copy(dy, dz, bytes, (int)std::min<size_t>(8192, (bytes + 16383) / 16384), stream);
    if (e != hipSuccess) return hip_fail(e, fn);
  }
  if (product) {
    W4Epilogue ep;
    ep.aux = dy;
    ep.act = act;
    const bool split = plan_w4_gemm(M, P, d).partial_bytes != 0;
    uint32_t* cnt = split ? (uint32_t*)ws : nullptr;
    float* part = split ? (float*)(ws + kDecodeCounterBytes) : nullptr;
    auto launch = gated ? launch_w4_gemm_gated_grad : launch_w4_gemm_act_grad;
    if (w4_tiles_fit(M, P, d))
      e = launch_w4_tiles(gated ? kEpiGatedGrad : kEpiActGrad, x, qweight, scales, zeros, bias, dz, M, N, d, group, ep,
                          stream);
    else
      e = launch(x, qweight, scales, zeros, bias, dz, M, N, d, group, cnt, part, ep, stream);
    if (e != hipSuccess) return hip_fail(e, fn);
  }
  if (dx) {
    e = launch_w4_input_grad(product ? dz : dy, qweight, scales, zeros, dx, M, P, d, group, (uint32_t*)ws, ws + first,
                             stream);
    if (e != hipSuccess) return hip_fail(e, fn);
  }
  return PARO_OK;
}

size_t backward_size(bool gated, int64_t M, int64_t N, int64_t d, int32_t act) {
  // (sizes that the call refuses: 0; the plans below count whole tiles of both)
  if (M <= 0 || N <= 0 || d <= 0 || M > (int64_t(1) << 30) || N > (int64_t(1) << 21) || d > (int64_t(1) << 22) ||
      N % 16 || d % 128)
    return 0;
  const int64_t P = gated ? 2 * N : N;
  return product_scratch(gated || act != PARO_ACT_NONE, M, P, d) + input_grad_scratch_bytes(M, P, d);
}

}  // namespace
}  // namespace paro

using namespace paro;

extern "C" {

int paro_w4_linear_act(const paro_rotation* r, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                       const uint8_t* zeros, const uint16_t* bias, const uint16_t* residual, int32_t act, uint16_t* y,
                       int64_t M, int64_t N, int64_t d, int32_t group, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  return run_forward("paro_w4_linear_act", kEpiAct, r, x, qweight, scales, zeros, bias, residual, act, y, M, N, d,
                     group, workspace, workspace_bytes, stream);
}

size_t paro_w4_gated_workspace_size(const paro_rotation* r, int64_t M, int64_t N, int64_t d) {
  if (N <= 0 || N > (int64_t(1) << 29)) return 0;
  return paro_w4_linear_workspace_size(r, M, 2 * N, d);
}

int paro_w4_gated(const paro_rotation* r, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                  const uint8_t* zeros, const uint16_t* bias, int32_t act, uint16_t* y, int64_t M, int64_t N,
                  int64_t d, int32_t group, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return run_forward("paro_w4_gated", kEpiGated, r, x, qweight, scales, zeros, bias, nullptr, act, y, M, N, d, group,
                     workspace, workspace_bytes, stream);
}

size_t paro_w4_linear_act_backward_workspace_size(int64_t M, int64_t N, int64_t d, int32_t act) {
  return backward_size(false, M, N, d, act);
}

int paro_w4_linear_act_backward(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                                const uint8_t* zeros, const uint16_t* bias, int32_t act, const uint16_t* dy,
                                uint16_t* dz, uint16_t* dx, int64_t M, int64_t N, int64_t d, int32_t group,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return run_backward("paro_w4_linear_act_backward", false, x, qweight, scales, zeros, bias, act, dy, dz, dx, M, N, d,
                      group, workspace, workspace_bytes, stream);
}

size_t paro_w4_gated_backward_workspace_size(int64_t M, int64_t N, int64_t d) {
  return backward_size(true, M, N, d, PARO_ACT_SILU);
}

int paro_w4_gated_backward(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                           const uint16_t* bias, int32_t act, const uint16_t* dy, uint16_t* dz, uint16_t* dx,
                           int64_t M, int64_t N, int64_t d, int32_t group, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  return run_backward("paro_w4_gated_backward", true, x, qweight, scales, zeros, bias, act, dy, dz, dx, M, N, d,
                      group, workspace, workspace_bytes, stream);
}

}  // extern "C"

// The launches of one step, fixed when the plan is made; a step fills in its
// scalars. Short lists as kernel arguments (lists), long ones as parts of the
// device table (first tensor and first chunk of each launch).
struct paro_adamw {
  int32_t param_type = 0, grad_type = 0;
  bool eight = false;
  void *m = nullptr, *v = nullptr;
  float *ms = nullptr, *vs = nullptr;
  std::vector<AdamwLaunch> lists;
  struct Part {
    size_t tensor0, chunk0;
  };
  std::vector<Part> parts;
  std::vector<uint32_t> chunks;  // of each launch
  AdamwTensor* d_tensors = nullptr;
  uint32_t* d_of_chunk = nullptr;
  ~paro_adamw() {
    if (d_tensors) (void)hipFree(d_tensors);
    if (d_of_chunk) (void)hipFree(d_of_chunk);
  }
};

namespace paro {
namespace {

int64_t type_bytes(int32_t t) { return t == PARO_TYPE_F32 ? 4 : 2; }
bool known_type(int32_t t) { return t >= PARO_TYPE_F32 && t <= PARO_TYPE_BF16; }

// Total blocks of 256 moments, or -1 for a bad list
int64_t total_blocks(int32_t count, const int64_t* n) {
  if (count < 0 || (count > 0 && !n)) return -1;
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (n[i] < 0 || n[i] > (int64_t(1) << 38)) return -1;
    total += (n[i] + 255) / 256;
    if (total > int64_t(UINT32_MAX)) return -1;
  }
  return total;
}

}  // namespace
}  // namespace paro

extern "C" {

int64_t paro_adamw_moments(int32_t count, const int64_t* n) {
  const int64_t blocks = total_blocks(count, n);
  return blocks < 0 ? -1 : blocks * 256;
}

int paro_adamw_create(int32_t count, const int64_t* n, void* const* params, int32_t param_type,
                      const void* const* grads, int32_t grad_type, int32_t state_bits, void* m, void* v,
                      float* m_scale, float* v_scale, paro_adamw** out) {
  if (!out) return fail(PARO_ERR_NULL, "paro_adamw_create: out is NULL");
  *out = nullptr;
  if (!known_type(param_type) || !known_type(grad_type))
    return fail(PARO_ERR_VALUE, "paro_adamw_create: unknown parameter or gradient type");
  if (state_bits != 32 && state_bits != 8)
    return fail(PARO_ERR_UNSUPPORTED, "paro_adamw_create: state_bits must be 32 or 8");
  const int64_t blocks = total_blocks(count, n);
  if (blocks < 0) return fail(PARO_ERR_SHAPE, "paro_adamw_create: bad tensor sizes");
  const bool eight = state_bits == 8;
  if (count > 0 && (!params || !grads)) return fail(PARO_ERR_NULL, "paro_adamw_create: NULL list");
  if (blocks > 0 && (!m || !v || (eight && (!m_scale || !v_scale))))
    return fail(PARO_ERR_NULL, "paro_adamw_create: NULL moments or scales");
  if (!aligned16(m) || !aligned16(v) || ((uintptr_t)m_scale & 3) || ((uintptr_t)v_scale & 3))
    return fail(PARO_ERR_ALIGN, "paro_adamw_create: moments must be 16-byte aligned, scales 4-byte");
  try {
    // every range that a step writes, to refuse two that overlap: a value
    // would be stepped twice, in no fixed order
    std::vector<std::pair<uintptr_t, uintptr_t>> written;
    auto add = [&](const void* p, int64_t bytes) {
      if (bytes > 0) written.emplace_back((uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes);
    };
    const uintptr_t pmask = (uintptr_t)type_bytes(param_type) - 1, gmask = (uintptr_t)type_bytes(grad_type) - 1;
    for (int32_t i = 0; i < count; ++i) {
      if (n[i] == 0) continue;
      if (!params[i] || !grads[i]) return fail(PARO_ERR_NULL, "paro_adamw_create: NULL tensor");
      if (((uintptr_t)params[i] & pmask) || ((uintptr_t)grads[i] & gmask))
        return fail(PARO_ERR_ALIGN, "paro_adamw_create: a tensor is not aligned to its type");
      add(params[i], n[i] * type_bytes(param_type));
    }
    add(m, blocks * 256 * (eight ? 1 : 4));
    add(v, blocks * 256 * (eight ? 1 : 4));
    if (eight) {
      add(m_scale, blocks * 4);
      add(v_scale, blocks * 4);
    }
    std::sort(written.begin(), written.end());
    for (size_t i = 1; i < written.size(); ++i)
      if (written[i].first < written[i - 1].second)
        return fail(PARO_ERR_VALUE, "paro_adamw_create: parameters or moments overlap");
    for (int32_t i = 0; i < count; ++i) {
      const uintptr_t g0 = (uintptr_t)grads[i], g1 = g0 + (uintptr_t)(n[i] * type_bytes(grad_type));
      if (n[i] == 0) continue;
      auto it = std::upper_bound(written.begin(), written.end(), std::make_pair(g0, UINTPTR_MAX));
      if ((it != written.begin() && (it - 1)->second > g0) || (it != written.end() && it->first < g1))
        return fail(PARO_ERR_VALUE, "paro_adamw_create: a gradient overlaps what the step writes");
    }

    // the pieces of each launch (a very large tensor takes several)
    constexpr uint32_t kMostChunks = 1u << 22;
    std::vector<std::vector<AdamwTensor>> launches(1);
    std::unique_ptr<paro_adamw> h(new paro_adamw());
    uint32_t chunk = 0, block = 0;
    for (int32_t i = 0; i < count; ++i) {
      for (int64_t at = 0; at < n[i];) {
        if (chunk == kMostChunks) {
          h->chunks.push_back(chunk);
          launches.emplace_back();
          chunk = 0;
        }
        AdamwTensor t;
        t.p = (char*)params[i] + at * type_bytes(param_type);
        t.g = (const char*)grads[i] + at * type_bytes(grad_type);
        t.n = std::min(n[i] - at, (int64_t)(kMostChunks - chunk) * kAdamChunk);
        t.chunk0 = chunk;
        t.block0 = block;
        chunk += (uint32_t)((t.n + kAdamChunk - 1) / kAdamChunk);
        block += (uint32_t)((t.n + 255) / 256);
        at += t.n;
        launches.back().push_back(t);
      }
    }
    h->chunks.push_back(chunk);
    h->param_type = param_type;
    h->grad_type = grad_type;
    h->eight = eight;
    h->m = m;
    h->v = v;
    h->ms = m_scale;
    h->vs = v_scale;
    bool table = false;
    for (const auto& l : launches) table = table || l.size() > (size_t)kAdamTensors;
    if (!table) {
      for (const auto& l : launches) {
        AdamwLaunch a;
        std::memset(&a, 0, sizeof(a));
        a.count = (int32_t)l.size();
        std::copy(l.begin(), l.end(), a.t);
        h->lists.push_back(a);
      }
    } else {
      std::vector<AdamwTensor> all;
      std::vector<uint32_t> of_chunk;
      for (const auto& l : launches) {
        h->parts.push_back({all.size(), of_chunk.size()});
        for (size_t k = 0; k < l.size(); ++k)
          of_chunk.insert(of_chunk.end(), (size_t)((l[k].n + kAdamChunk - 1) / kAdamChunk), (uint32_t)k);
        all.insert(all.end(), l.begin(), l.end());
      }
      hipError_t e = hipMalloc((void**)&h->d_tensors, all.size() * sizeof(AdamwTensor));
      if (e == hipSuccess) e = hipMalloc((void**)&h->d_of_chunk, of_chunk.size() * sizeof(uint32_t));
      if (e == hipSuccess)
        e = hipMemcpy(h->d_tensors, all.data(), all.size() * sizeof(AdamwTensor), hipMemcpyHostToDevice);
      if (e == hipSuccess)
        e = hipMemcpy(h->d_of_chunk, of_chunk.data(), of_chunk.size() * sizeof(uint32_t), hipMemcpyHostToDevice);
      if (e != hipSuccess) return hip_fail(e, "paro_adamw_create: table of tensors");
    }
    *out = h.release();
  } catch (const std::exception& e) {
    return fail(PARO_ERR_UNSUPPORTED, std::string("paro_adamw_create: ") + e.what());
  }
  return PARO_OK;
}

void paro_adamw_destroy(paro_adamw* h) { delete h; }

int paro_adamw_step(const paro_adamw* h, int64_t step, double lr, double beta1, double beta2, double eps,
                    double weight_decay, hipStream_t stream) {
  if (!h) return fail(PARO_ERR_NULL, "paro_adamw_step: NULL plan");
  if (step < 1) return fail(PARO_ERR_VALUE, "paro_adamw_step: step must be at least 1");
  if (!std::isfinite(lr) || lr < 0 || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) ||
      !((float)eps > 0 && std::isfinite((float)eps)) || !std::isfinite(weight_decay) || weight_decay < 0)
    return fail(PARO_ERR_VALUE, "paro_adamw_step: lr >= 0, 0 <= beta < 1, eps > 0, weight_decay >= 0, all finite");
  const double c1 = 1.0 - std::pow(beta1, (double)step), c2 = 1.0 - std::pow(beta2, (double)step);
  AdamwScalars sc;
  sc.m = h->m;
  sc.v = h->v;
  sc.ms = h->ms;
  sc.vs = h->vs;
  sc.b1 = (float)beta1;
  sc.c1 = (float)(1.0 - beta1);
  sc.b2 = (float)beta2;
  sc.c2 = (float)(1.0 - beta2);
  sc.keep = (float)(1.0 - lr * weight_decay);
  sc.rate = (float)(lr / c1);
  sc.root = (float)(1.0 / std::sqrt(c2));
  sc.eps = (float)eps;
  if (!std::isfinite(sc.keep) || !std::isfinite(sc.rate))
    return fail(PARO_ERR_VALUE, "paro_adamw_step: lr or lr * weight_decay too large for fp32");
  for (size_t i = 0; i < h->chunks.size(); ++i) {
    hipError_t e;
    if (h->parts.empty()) {
      AdamwLaunch a = h->lists[i];
      a.s = sc;
      e = launch_adamw(a, h->chunks[i], h->param_type, h->grad_type, h->eight, stream);
    } else {
      const AdamwTable a = {sc, h->d_tensors + h->parts[i].tensor0, h->d_of_chunk + h->parts[i].chunk0};
      e = launch_adamw(a, h->chunks[i], h->param_type, h->grad_type, h->eight, stream);
    }
    if (e != hipSuccess) return hip_fail(e, "paro_adamw_step launch");
  }
  return PARO_OK;
}

}  // extern "C"
