// C ABI of the mixture-of-experts operators and the distillation loss
// (declarations and argument contracts in include/paro.h).
#include <algorithm>
#include <cmath>
#include <string>
#include <vector>

#include "paro_internal.h"
#include "w4_epilogue.h"

namespace paro {
namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int fail(int status, const std::string& msg) {
  set_error(msg);
  return status;
}

int hip_fail(hipError_t e, const char* what) { return fail(PARO_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e)); }

size_t a256(size_t b) { return (b + 255) & ~(size_t)255; }

bool known_type(int32_t t) { return t >= PARO_TYPE_F32 && t <= PARO_TYPE_BF16; }

// Limits under which every launch has fewer than 2^32 lanes in its grid: pairs of a call;
// pairs, and experts, times the wider of an expert's sides (a tile of the products has
// 2048 values by 256 lanes or more, and every expert may end in one that is nearly
// empty); rows of the loss.
constexpr int64_t kMaxPairs = (int64_t(1) << 24) - 1, kMaxRowValues = int64_t(1) << 34,
                  kMaxStack = int64_t(1) << 27, kMaxLossRows = (int64_t(1) << 22) - 1;

bool good_experts(int64_t M, int32_t E, int32_t k) {
  return M >= 0 && E >= 1 && k >= 1 && k <= E;
}
// *noop: no tokens
int check_experts(const std::string& f, int64_t M, int32_t E, int32_t k, bool* noop) {
  if (!good_experts(M, E, k)) return fail(PARO_ERR_SHAPE, f + ": M >= 0 and 1 <= k <= E");
  if (E > kExpertsMax || k > kExpertsMaxK)
    return fail(PARO_ERR_UNSUPPORTED, f + ": at most 1024 experts, 16 of them for a token");
  if (M > kMaxPairs / k) return fail(PARO_ERR_UNSUPPORTED, f + ": fewer than 2^24 pairs of token and expert");
  *noop = M == 0;
  return PARO_OK;
}

int check_workspace(const std::string& f, size_t need, const void* ws, size_t bytes) {
  if (need && (!ws || bytes < need))
    return fail(PARO_ERR_WORKSPACE, f + ": workspace missing or smaller than the size reported for these arguments");
  if (!aligned(ws, 256)) return fail(PARO_ERR_ALIGN, f + ": workspace must be 256-byte aligned");
  return PARO_OK;
}

// The checks that the experts' products share: the routing, the weight stack of
// P rows an expert, and y, the call's output. wants: whether the weights of the
// pairs are used, and tokens: the widest row that is read or written by token.
int check_product(const std::string& f, const paro_routing* r, const void* x, const uint8_t* qweight,
                  const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, const void* y, int64_t P,
                  int64_t d, int32_t group, bool wants, int64_t by_token, ExpertRouting* t, bool* noop) {
  if (!r) return fail(PARO_ERR_NULL, f + ": routing is NULL");
  const int st = check_experts(f, r->M, r->E, r->k, noop);
  if (st != PARO_OK) return st;
  if (group != 64 && group != 128 && group != 256)
    return fail(PARO_ERR_UNSUPPORTED, f + ": group must be 64, 128 or 256");
  if (P <= 0 || P % 16 || d <= 0 || d % 128 || d % group)
    return fail(PARO_ERR_SHAPE, f + ": N % 16 == 0, d % 128 == 0 and d % group == 0");
  if (P > (int64_t(1) << 21) || d > (int64_t(1) << 21) || P * d >= (int64_t(1) << 31))
    return fail(PARO_ERR_UNSUPPORTED, f + ": an expert's weights: at most 2^21 rows or channels, fewer than 2^31 values");
  if (r->M * by_token >= (int64_t(1) << 30))
    return fail(PARO_ERR_UNSUPPORTED, f + ": tokens times their channels must be below 2^30");
  if (r->M * r->k * std::max(P, d) >= kMaxRowValues || r->E * std::max(P, d) >= kMaxStack)
    return fail(PARO_ERR_UNSUPPORTED, f + ": pairs times channels must be below 2^34, experts times channels below 2^27");
  if (*noop) return PARO_OK;
  if (!x || !qweight || !scales || !zeros || !y) return fail(PARO_ERR_NULL, f + ": NULL tensor");
  if (!r->offsets || !r->order || !r->place || !r->ids || (wants && !r->weights))
    return fail(PARO_ERR_NULL, f + ": NULL table in the routing");
  if (!aligned(x, 16) || !aligned(qweight, 16) || !aligned(scales, 16) || !aligned(zeros, 16) || !aligned(bias, 16) ||
      !aligned(y, 16))
    return fail(PARO_ERR_ALIGN, f + ": tensors must be 16-byte aligned");
  if (!aligned(r->offsets, 4) || !aligned(r->order, 4) || !aligned(r->place, 4) || !aligned(r->ids, 4) ||
      !aligned(r->weights, 4))
    return fail(PARO_ERR_ALIGN, f + ": the routing's tables must be 4-byte aligned");
  *t = {(int)r->M, r->E, r->k, (int)(r->M * r->k), r->ids, r->offsets, r->order, r->place, r->weights};
  return PARO_OK;
}

bool good_sizes(int64_t M, int32_t E, int32_t k, int64_t P, int64_t d) {
  return good_experts(M, E, k) && M > 0 && E <= kExpertsMax && k <= kExpertsMaxK && M <= kMaxPairs / k && P > 0 &&
         P % 16 == 0 && d > 0 && d % 128 == 0 && P <= (int64_t(1) << 21) && d <= (int64_t(1) << 21) &&
         P * d < (int64_t(1) << 31) && M * k * std::max(P, d) < kMaxRowValues && E * std::max(P, d) < kMaxStack;
}

ExpertRouting sizes_only(int64_t M, int32_t E, int32_t k) {
  return {(int)M, E, k, (int)(M * k), nullptr, nullptr, nullptr, nullptr, nullptr};
}

size_t grad_bytes(const ExpertRouting& t, int64_t P, int64_t d, bool share) {
  if (!experts_grad_wide_fit(t, P, d, share)) return a256((size_t)experts_grad_rows_splits(t, P, d) * t.R * d * 4);
  return a256(share ? experts_grad_dots(t, d) : (size_t)experts_grad_splits(t, P, d) * t.R * d * 4);
}

// The most that grad_bytes asks for up to M tokens, so that a workspace for the
// largest batch serves every smaller one: its size grows with M but where the rules
// choose another way, so that the last M before each step, and M itself, are looked at.
size_t grad_peak(int64_t M, int32_t E, int32_t k, int64_t P, int64_t d, bool share) {
  std::vector<int64_t> rows;
  rows.reserve(64);
  experts_grad_rows_steps(E, d, rows);
  experts_grad_wide_steps(E, d, rows);
  size_t most = grad_bytes(sizes_only(M, E, k), P, d, share);
  for (const int64_t r : rows)
    if (r / k >= 1 && r / k < M) most = std::max(most, grad_bytes(sizes_only(r / k, E, k), P, d, share));
  return most;
}

bool known_act(int32_t act) { return act >= PARO_ACT_NONE && act <= PARO_ACT_RELU; }

}  // namespace
}  // namespace paro

using namespace paro;

extern "C" {

size_t paro_experts_route_workspace_size(int64_t M, int32_t E, int32_t k) {
  if (!good_experts(M, E, k) || E > kExpertsMax || k > kExpertsMaxK || M > kMaxPairs / k) return 0;
  // (the most of any number of tokens up to M: chunks get larger behind these)
  size_t most = experts_route_scratch(M, E, k);
  for (const int64_t m : {int64_t(16384), int64_t(32768), int64_t(1) << 18})
    if (m < M) most = std::max(most, experts_route_scratch(m, E, k));
  return most;
}

int paro_experts_route(const void* logits, int32_t type, int64_t M, int32_t E, int32_t k, int32_t normalize,
                       int32_t* ids, float* weights, int32_t* offsets, int32_t* order, int32_t* place,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const std::string f("paro_experts_route");
  bool none = false;
  int st = check_experts(f, M, E, k, &none);
  if (st != PARO_OK) return st;
  if (!known_type(type)) return fail(PARO_ERR_VALUE, f + ": unknown type of the logits");
  if (!offsets || (!none && (!logits || !ids || !weights || !order || !place)))
    return fail(PARO_ERR_NULL, f + ": NULL tensor");
  if (!aligned(logits, type == PARO_TYPE_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(offsets, 4) || !aligned(order, 4) || !aligned(place, 4))
    return fail(PARO_ERR_ALIGN, f + ": a tensor is not aligned to its type");
  if ((st = check_workspace(f, experts_route_scratch(M, E, k), workspace, workspace_bytes)) != PARO_OK) return st;
  // (no tokens: every expert's rows are empty)
  const hipError_t e = none ? launch_fill_zero((float*)offsets, E + 1, stream)
                            : launch_experts_route(logits, type, M, E, k, normalize != 0, ids, weights, offsets, order,
                                                   place, workspace, stream);
  return e == hipSuccess ? PARO_OK : hip_fail(e, "paro_experts_route");
}

int paro_experts_sort(const int32_t* ids, int64_t M, int32_t E, int32_t k, int32_t* offsets, int32_t* order,
                      int32_t* place, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const std::string f("paro_experts_sort");
  bool none = false;
  int st = check_experts(f, M, E, k, &none);
  if (st != PARO_OK) return st;
  if (!offsets || (!none && (!ids || !order || !place))) return fail(PARO_ERR_NULL, f + ": NULL tensor");
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(place, 4))
    return fail(PARO_ERR_ALIGN, f + ": a tensor is not aligned to its type");
  if ((st = check_workspace(f, experts_route_scratch(M, E, k), workspace, workspace_bytes)) != PARO_OK) return st;
  const hipError_t e = none ? launch_fill_zero((float*)offsets, E + 1, stream)
                            : launch_experts_route(nullptr, 0, M, E, k, 0, const_cast<int32_t*>(ids), nullptr, offsets,
                                                   order, place, workspace, stream);
  return e == hipSuccess ? PARO_OK : hip_fail(e, "paro_experts_sort");
}

int paro_experts_route_backward(const void* logits, int32_t type, int64_t M, int32_t E, int32_t k, int32_t normalize,
                                const int32_t* ids, const float* weights, const float* dweights, void* dlogits,
                                hipStream_t stream) {
  const std::string f("paro_experts_route_backward");
  bool none = false;
  const int st = check_experts(f, M, E, k, &none);
  if (st != PARO_OK) return st;
  if (!known_type(type)) return fail(PARO_ERR_VALUE, f + ": unknown type of the logits");
  if (none) return PARO_OK;
  if ((!normalize && !logits) || !ids || !weights || !dweights || !dlogits)
    return fail(PARO_ERR_NULL, f + ": NULL tensor");
  const uintptr_t size = type == PARO_TYPE_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(dweights, 4))
    return fail(PARO_ERR_ALIGN, f + ": a tensor is not aligned to its type");
  const hipError_t e = launch_experts_route_backward(logits, type, M, E, k, normalize != 0, ids, weights, dweights,
                                                     dlogits, stream);
  return e == hipSuccess ? PARO_OK : hip_fail(e, "paro_experts_route_backward");
}

size_t paro_w4_experts_gated_workspace_size(int64_t, int32_t, int32_t, int64_t, int64_t) { return 0; }

int paro_w4_experts_gated(const paro_routing* routing, const uint16_t* x, const uint8_t* qweight,
                          const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, int32_t act,
                          uint16_t* h, int64_t N, int64_t d, int32_t group, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
  const std::string f("paro_w4_experts_gated");
  if (!known_act(act)) return fail(PARO_ERR_VALUE, f + ": unknown activation");
  if (N > (int64_t(1) << 20)) return fail(PARO_ERR_UNSUPPORTED, f + ": at most 2^21 weight rows");
  if (N % 16) return fail(PARO_ERR_SHAPE, f + ": N must be a positive multiple of 16");
  ExpertRouting t;
  bool none = false;
  int st = check_product(f, routing, x, qweight, scales, zeros, bias, h, 2 * N, d, group, false, d, &t, &none);
  if (st != PARO_OK || none) return st;
  if ((st = check_workspace(f, 0, workspace, workspace_bytes)) != PARO_OK) return st;
  W4Epilogue ep;
  ep.act = act;
  const hipError_t e = launch_w4_experts(kEpiGated, t, x, qweight, scales, zeros, bias, h, N, d, group, ep, stream);
  return e == hipSuccess ? PARO_OK : hip_fail(e, "paro_w4_experts_gated");
}

size_t paro_w4_experts_combine_workspace_size(int64_t M, int32_t E, int32_t k, int64_t N, int64_t d) {
  return good_sizes(M, E, k, N, d) ? a256((size_t)M * k * N * 4) : 0;
}

int paro_w4_experts_combine(const paro_routing* routing, const uint16_t* h, const uint8_t* qweight,
                            const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias,
                            const uint16_t* residual, uint16_t* y, int64_t N, int64_t d, int32_t group,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const std::string f("paro_w4_experts_combine");
  ExpertRouting t;
  bool none = false;
  int st = check_product(f, routing, h, qweight, scales, zeros, bias, y, N, d, group, true, N, &t, &none);
  if (st != PARO_OK || none) return st;
  if (!aligned(residual, 16)) return fail(PARO_ERR_ALIGN, f + ": residual must be 16-byte aligned");
  const size_t need = paro_w4_experts_combine_workspace_size(t.M, t.E, t.k, N, d);
  if ((st = check_workspace(f, need, workspace, workspace_bytes)) != PARO_OK) return st;
  hipError_t e = launch_w4_experts(kEpiShare, t, h, qweight, scales, zeros, bias, workspace, N, d, group,
                                         W4Epilogue{}, stream);
  if (e == hipSuccess) e = launch_experts_sum(t, (const float*)workspace, 1, residual, y, N, stream);
  return e == hipSuccess ? PARO_OK : hip_fail(e, "paro_w4_experts_combine");
}

size_t paro_w4_experts_gated_backward_workspace_size(int64_t M, int32_t E, int32_t k, int64_t N, int64_t d) {
  if (N > (int64_t(1) << 20) || !good_sizes(M, E, k, 2 * N, d) || N % 16) return 0;
  return grad_peak(M, E, k, 2 * N, d, false);
}

int paro_w4_experts_gated_backward(const paro_routing* routing, const uint16_t* x, const uint8_t* qweight,
                                   const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, int32_t act,
                                   const uint16_t* dh, uint16_t* dz, uint16_t* dx, int64_t N, int64_t d,
                                   int32_t group, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const std::string f("paro_w4_experts_gated_backward");
  if (!known_act(act)) return fail(PARO_ERR_VALUE, f + ": unknown activation");
  if (N > (int64_t(1) << 20)) return fail(PARO_ERR_UNSUPPORTED, f + ": at most 2^21 weight rows");
  if (N % 16) return fail(PARO_ERR_SHAPE, f + ": N must be a positive multiple of 16");
  ExpertRouting t;
  bool none = false;
  int st = check_product(f, routing, x, qweight, scales, zeros, bias, dz, 2 * N, d, group, false, d, &t, &none);
  if (st != PARO_OK || none) return st;
  if (!dh) return fail(PARO_ERR_NULL, f + ": NULL tensor");
  if (!aligned(dh, 16) || !aligned(dx, 16)) return fail(PARO_ERR_ALIGN, f + ": dh and dx must be 16-byte aligned");
  const size_t need = dx ? grad_bytes(t, 2 * N, d, false) : 0;
  if ((st = check_workspace(f, need, workspace, workspace_bytes)) != PARO_OK) return st;
  W4Epilogue ep;
  ep.aux = dh;
  ep.act = act;
  // dX' is the product of dZ as it is returned, rounded to fp16: half a step, 2^-11, of
  // each term, at random, which the sum keeps beside its own rounding (2.9e-4 of the
  // norm against 2.1e-4 for an operand in fp32, that would take the matrix cores twice).
  hipError_t e = launch_w4_experts(kEpiGatedGrad, t, x, qweight, scales, zeros, bias, dz, N, d, group, ep, stream);
  if (e == hipSuccess && dx) {
    const bool wide = experts_grad_wide_fit(t, 2 * N, d, false);
    const int splits = wide ? experts_grad_splits(t, 2 * N, d) : experts_grad_rows_splits(t, 2 * N, d);
    float* part = (float*)workspace;
    e = wide ? launch_w4_experts_grad_part(t, dz, qweight, scales, zeros, part, 2 * N, d, group, stream)
             : launch_w4_experts_grad_rows(t, false, dz, qweight, scales, zeros, part, 2 * N, d, group, stream);
    if (e == hipSuccess) e = launch_experts_sum(t, (const float*)workspace, splits, nullptr, dx, d, stream);
  }
  return e == hipSuccess ? PARO_OK : hip_fail(e, "paro_w4_experts_gated_backward");
}

size_t paro_w4_experts_combine_backward_workspace_size(int64_t M, int32_t E, int32_t k, int64_t N, int64_t d) {
  return good_sizes(M, E, k, N, d) ? grad_peak(M, E, k, N, d, true) : 0;
}

int paro_w4_experts_combine_backward(const paro_routing* routing, const uint16_t* h, const uint8_t* qweight,
                                     const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias,
                                     const uint16_t* dy, uint16_t* dh, float* dweights, int64_t N, int64_t d,
                                     int32_t group, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const std::string f("paro_w4_experts_combine_backward");
  ExpertRouting t;
  bool none = false;
  int st = check_product(f, routing, h, qweight, scales, zeros, bias, dh, N, d, group, true, N, &t, &none);
  if (st != PARO_OK || none) return st;
  if (!dy || !dweights) return fail(PARO_ERR_NULL, f + ": NULL tensor");
  if (!aligned(dy, 16) || !aligned(dweights, 4))
    return fail(PARO_ERR_ALIGN, f + ": dy must be 16-byte aligned, dweights 4-byte");
  const size_t need = grad_bytes(t, N, d, true);
  if ((st = check_workspace(f, need, workspace, workspace_bytes)) != PARO_OK) return st;
  float* part = (float*)workspace;
  hipError_t e;
  if (experts_grad_wide_fit(t, N, d, true)) {
    e = launch_w4_experts_grad_share(t, dy, qweight, scales, zeros, part, h, dh, N, d, group, stream);
    if (e == hipSuccess)
      e = launch_experts_dots(t, part, (int)(experts_grad_dots(t, d) / 4 / t.R), dy, bias, dweights, N, stream);
  } else {
    e = launch_w4_experts_grad_rows(t, true, dy, qweight, scales, zeros, part, N, d, group, stream);
    if (e == hipSuccess)
      e = launch_experts_share_grad(t, part, experts_grad_rows_splits(t, N, d), h, dy, bias, dh, dweights, N, d, stream);
  }
  return e == hipSuccess ? PARO_OK : hip_fail(e, "paro_w4_experts_combine_backward");
}

int paro_distill_loss(const void* z, int32_t z_type, const void* values, int32_t value_type, const int32_t* index,
                      const float* lse, const float* row_weight, int64_t M, int64_t V, int64_t K, double temperature,
                      double grad_scale, float* loss, void* dz, hipStream_t stream) {
  const std::string f("paro_distill_loss");
  if (!known_type(z_type) || !known_type(value_type)) return fail(PARO_ERR_VALUE, f + ": unknown type");
  if (M < 0 || V < 1 || K < 1) return fail(PARO_ERR_SHAPE, f + ": M >= 0, V >= 1 and K >= 1");
  if (M > kMaxLossRows || V > (int64_t(1) << 20) || K > 1024)
    return fail(PARO_ERR_UNSUPPORTED, f + ": fewer than 2^22 rows, at most 2^20 logits and 1024 of the teacher's");
  const float T = (float)temperature, scale = (float)grad_scale;
  // (log2(e) / T is the factor of the kernel's exponents)
  if (!(T > 0) || !std::isfinite(T) || !std::isfinite((float)(1.4426950408889634 / (double)T)) || !std::isfinite(scale))
    return fail(PARO_ERR_VALUE, f + ": temperature must be positive and above 4.3e-39, and it and grad_scale finite in fp32");
  if (M == 0) return PARO_OK;
  if (!z || !values || !index || !loss) return fail(PARO_ERR_NULL, f + ": NULL tensor");
  if (!aligned(z, 16) || !aligned(dz, 16) || !aligned(values, value_type == PARO_TYPE_F32 ? 4 : 2) ||
      !aligned(index, 4) || !aligned(lse, 4) || !aligned(row_weight, 4) || !aligned(loss, 4))
    return fail(PARO_ERR_ALIGN, f + ": z and dz must be 16-byte aligned, the others to their type");
  const DistillArgs a = {z, values, index, lse, row_weight, loss, dz, M, (int)V, (int)K, T, scale};
  const hipError_t e = launch_distill(a, z_type, value_type, stream);
  return e == hipSuccess ? PARO_OK : hip_fail(e, "paro_distill_loss");
}

}  // extern "C"
