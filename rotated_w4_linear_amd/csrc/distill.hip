// gfx950 kernel of the distillation loss from a teacher's top logits, with its
// gradient: for every row, with q = softmax(z / T) over V and the teacher's
// entries i (logit t_i at index j_i),
//   p_i = exp(t_i / T) / sum_i exp(t_i / T), or exp(t_i / T - lse) and P = the
//         rest of the teacher's mass (>= 0), Q = the student's outside the entries,
//   L   = w T^2 [sum_i p_i (log p_i - log q_i) + P (log P - log Q)],
//   dz_j = w T (A q_j - p_j), and outside the entries w T q_j (A - P / Q),
// A = sum p + P (1 but for rounding).
//
// One workgroup per row. A first pass over z takes the running maximum and sum
// of exponentials (leaving the entries out, by a bitmap of V bits in LDS, where
// the rest is a class of its own); the entries are done in fp64, and the sum of
// everything is the rest's plus the entries': where teacher and student agree,
// L is a small difference, and an error of the rest's sum then enters by Q - P
// only. A second pass writes the gradient. NV > 0: the row stays in registers
// between the passes, 16 bytes NV times a lane; else it is read again.
#include "paro_internal.h"
#include "paro_types.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_inff();

// The VE values of 16 bytes, and back.
template <class T>
struct Vec {
  static constexpr int VE = 16 / sizeof(typename T::raw);
  static __device__ __forceinline__ float get(const u4& v, int i) {
    const uint32_t word = v[VE == 4 ? i : i >> 1];  // (a bit cast of the element itself takes the first one)
    if constexpr (VE == 4) return __builtin_bit_cast(float, word);
    else return T::value((typename T::raw)(word >> (16 * (i & 1))));
  }
  static __device__ __forceinline__ u4 put(const float* f) {
    u4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (VE == 4) o[i] = __builtin_bit_cast(uint32_t, f[i]);
      else o[i] = (uint32_t)T::pack(f[2 * i]) | (uint32_t)T::pack(f[2 * i + 1]) << 16;
    }
    return o;
  }
};

// Sum, or maximum, over the workgroup, in a fixed order; every thread has it.
template <int NT, class V, class Op>
__device__ __forceinline__ V block_reduce(V v, V* red, Op op) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v = op(v, (V)__shfl_xor(v, s));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) v = op(v, red[i]);
  return v;
}

template <class Z, class TV, int NT, int NV>
__global__ __launch_bounds__(NT) void distill_kernel(DistillArgs a) {
  typedef typename Z::raw raw;
  constexpr int VE = Vec<Z>::VE;
  __shared__ double red[NT / 64];
  __shared__ int any_twice;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  double* p = (double*)dyn;                // [K]: p_i, then what the gradient at j_i is
  int* index = (int*)(p + a.K);            // [K], -1: no entry
  uint32_t* bits = (uint32_t*)(index + a.K);  // V bits and 8 (the words past K even are 4-byte aligned)
  const int tid = threadIdx.x, V = a.V, K = a.K;
  const int64_t m = blockIdx.x;
  const raw* z = (const raw*)a.z + m * V;
  raw* dz = a.dz ? (raw*)a.dz + m * V : nullptr;
  const float w = a.weight ? a.weight[m] : 1.0f;
  // 16-byte vectors from the first aligned element on; the elements before and
  // behind them one by one. Element j has bit j + shift: a vector's lie in one byte.
  const int head = min(V, (int)((16 - ((uintptr_t)z & 15)) & 15) / (int)sizeof(raw));
  const int nvec = (V - head) / VE, tail0 = head + nvec * VE, shift = (VE - head % VE) % VE;
  const int vbase = (head + shift) / VE;  // the first vector, in units of VE bits

  auto zeros = [&]() {
    if (dz) {
      for (int j = tid; j < head; j += NT) dz[j] = (raw)0;
      for (int v = tid; v < nvec; v += NT) *(u4*)(dz + head + v * VE) = u4{0u, 0u, 0u, 0u};
      for (int j = tail0 + tid; j < V; j += NT) dz[j] = (raw)0;
    }
    if (tid == 0) a.loss[m] = 0.0f;
  };
  if (w == 0.0f) return zeros();  // (a row that is left out: whatever it holds)

  // the teacher's entries
  const double it = 1.0 / (double)a.temperature;
  const int words = (V + VE + 31) / 32;
  for (int i = tid; i < words; i += NT) bits[i] = 0;
  if (tid == 0) any_twice = 0;
  __syncthreads();
  float tmax = -kInf;
  int entries = 0;
  for (int i = tid; i < K; i += NT) {
    const int j = a.index[m * K + i];
    const bool in = (uint32_t)j < (uint32_t)V;
    index[i] = in ? j : -1;
    if (!in) continue;
    const float t = TV::value(((const typename TV::raw*)a.values)[m * K + i]);
    if (t > -kInf || t != t) entries = 1;
    tmax = fmaxf(tmax, t);
    const uint32_t b = 1u << ((j + shift) & 31);
    if (atomicOr(&bits[(j + shift) >> 5], b) & b) any_twice = 1;
  }
  const bool rest = a.lse != nullptr;
  entries = __syncthreads_or(entries);
  if (!rest && !entries) return zeros();  // (a mask that leaves nothing of the teacher)
  if (!rest) tmax = block_reduce<NT>(tmax, (float*)red, [](float x, float y) { return fmaxf(x, y); });
  const double ref = rest ? (double)a.lse[m] : (double)tmax * it;
  double psum = 0.0;
  for (int i = tid; i < K; i += NT) {
    double v = 0.0;
    if (index[i] >= 0) v = exp((double)TV::value(((const typename TV::raw*)a.values)[m * K + i]) * it - ref);
    p[i] = v;
    psum += v;
  }
  auto add = [](double x, double y) { return x + y; };
  psum = block_reduce<NT>(psum, red, add);
  double P = 0.0, A = 1.0;
  if (rest) {
    P = fmax(1.0 - psum, 0.0);
    A = psum + P;
  }
  const double pscale = rest ? 1.0 : 1.0 / psum;

  // pass 1: maximum and sum
  const float c = (float)((double)kLog2e * it);
  float mx = -kInf, base = 0.0f, sum = 0.0f;  // base: mx, or 0 while nothing is above -inf
  auto taken = [&](int j) { return (bits[(j + shift) >> 5] >> ((j + shift) & 31)) & 1u; };
  auto more = [&](float hi) {
    if (hi > mx) {
      sum = mx > -kInf ? sum * __builtin_amdgcn_exp2f((mx - hi) * c) : 0.0f;
      base = mx = hi;
    }
  };
  auto one = [&](int j) {
    const float x = Z::value(z[j]);
    more(x);
    if (!rest || !taken(j)) sum += __builtin_amdgcn_exp2f((x - base) * c);
  };
  auto vec = [&](const u4& v, int at) {
    float x[VE], hi = -kInf;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      x[i] = Vec<Z>::get(v, i);
      hi = fmaxf(hi, x[i]);
    }
    more(hi);
    uint32_t out = 0;
    if (rest) out = bits[(vbase + at) * VE >> 5] >> ((vbase + at) * VE & 31) & ((1u << VE) - 1);
    float part = 0.0f;
    if (out == 0) {
#pragma unroll
      for (int i = 0; i < VE; ++i) part += __builtin_amdgcn_exp2f((x[i] - base) * c);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) part += (out >> i) & 1u ? 0.0f : __builtin_amdgcn_exp2f((x[i] - base) * c);
    }
    sum += part;
  };
  u4 held[NV > 0 ? NV : 1];
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (tid + k * NT < nvec) held[k] = *(const u4*)(z + head + (tid + k * NT) * VE);
  }
  for (int j = tid; j < head; j += NT) one(j);
  for (int j = tail0 + tid; j < V; j += NT) one(j);
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (tid + k * NT < nvec) vec(held[k], tid + k * NT);
  } else {
    for (int v = tid; v < nvec; v += NT) vec(*(const u4*)(z + head + v * VE), v);
  }
  // (a thread whose values are all -inf, or that has none: no sum)
  const float top = block_reduce<NT>(mx, (float*)red, [](float x, float y) { return fmaxf(x, y); });
  // NaN: fmax passes over it, the sum does not
  if (mx < top && sum == sum) sum = mx > -kInf ? sum * __builtin_amdgcn_exp2f((mx - top) * c) : 0.0f;
  const double left = block_reduce<NT>((double)sum, red, add);

  // the entries: p_i final, the student's mass there (each index once: the lowest
  // entry's, and its gradient with the masses of all entries of that index)
  const bool twice = any_twice != 0;
  double loss = 0.0, mass = 0.0;
  for (int i = tid; i < K; i += NT) {
    const int j = index[i];
    if (j < 0) continue;
    const double y = ((double)Z::value(z[j]) - (double)top) * it, pi = p[i] * pscale;
    if (pi != 0.0) loss += pi * (log(pi) - y);
    bool first = true;
    if (twice)
      for (int e = 0; e < i; ++e) first = first && index[e] != j;
    if (rest && first) mass += exp(y);
  }
  loss = block_reduce<NT>(loss, red, add);
  mass = block_reduce<NT>(mass, red, add);
  const double total = left + mass;  // (left holds everything without a class for the rest)
  if (tid == 0) {
    loss += A * log(total);
    if (P != 0.0) loss += P * (log(P) - log(left));
    a.loss[m] = (float)(loss * ((double)w * a.temperature * a.temperature));
  }
  if (!dz) return;
  const double g = (double)w * a.temperature * a.grad_scale;
  // the gradient at the entries, before anything of the row is overwritten (dz may be z)
  double mine[4];
  for (int i = tid, s = 0; i < K; i += NT, ++s) {
    const int j = index[i];
    double v = 0.0;
    if (j >= 0) {
      double all = p[i];
      if (twice) {
        all = 0.0;
        for (int e = 0; e < K; ++e) all += index[e] == j ? p[e] : 0.0;
      }
      v = (A * exp(((double)Z::value(z[j]) - (double)top) * it) / total - all * pscale) * g;
    }
    if (s == 0) mine[0] = v;
    else if (s == 1) mine[1] = v;
    else if (s == 2) mine[2] = v;
    else mine[3] = v;
  }
  __syncthreads();
  const float cf = (float)(g * (rest && left > 0.0 ? A / total - P / left : A / total));

  // pass 2 (a student without mass outside the entries has no gradient there)
  auto grad = [&](float x) { return __builtin_amdgcn_exp2f((x - top) * c) * cf; };
  auto grads = [&](const u4& v) {
    float f[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = grad(Vec<Z>::get(v, i));
    return Vec<Z>::put(f);
  };
  for (int j = tid; j < head; j += NT) dz[j] = Z::pack(grad(Z::value(z[j])));
  for (int j = tail0 + tid; j < V; j += NT) dz[j] = Z::pack(grad(Z::value(z[j])));
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (tid + k * NT < nvec) *(u4*)(dz + head + (tid + k * NT) * VE) = grads(held[k]);
  } else {
    for (int v = tid; v < nvec; v += NT) *(u4*)(dz + head + v * VE) = grads(*(const u4*)(z + head + v * VE));
  }
  __syncthreads();  // the entries' places have been written
  for (int i = tid, s = 0; i < K; i += NT, ++s) {
    const double v = s == 0 ? mine[0] : s == 1 ? mine[1] : s == 2 ? mine[2] : mine[3];
    if (index[i] >= 0) dz[index[i]] = Z::pack((float)v);
  }
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, int z_type, int value_type, hipStream_t stream) {
  with_type(z_type, [&](auto z) {
    with_type(value_type, [&](auto v) {
      typedef decltype(z) Z;
      typedef decltype(v) TV;
      const unsigned lds = (unsigned)(a.K * 12 + (a.V + Vec<Z>::VE + 31) / 32 * 4);
      hipLaunchKernelGGL((distill_kernel<Z, TV, 256, 0>), dim3((unsigned)a.M), dim3(256), lds, stream, a);
    });
  });
  return hipGetLastError();
}

}  // namespace paro
