// gfx950 kernels that join the experts of a token. The products leave their rows
// as fp32 sums, in expert order, and perhaps in pieces of the contraction: what a
// token's experts give is added in slot order and rounded once.
#include "paro_internal.h"
#include "w4_common.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

using namespace w4;

constexpr int kThreads = 256;

// y[m][n] = residual[m][n] + sum_s sum_p part[p][place[m][s]][n], four channels a
// lane. Bound by memory: k (splits) fp32 rows read per fp16 row written (2048 tokens,
// 4 rows of 2048 each: 76 MB in 13 us, in part from the memory-side cache).
__global__ __launch_bounds__(kThreads) void sum_kernel(ExpertRouting t, const float* __restrict__ part, int splits,
                                                       const uint16_t* residual, uint16_t* y, int N4) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t m = i / N4;
  if (m >= t.M) return;
  const int c = (int)(i - m * N4);
  f4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < t.k; ++s) {
    const int row = t.place[m * t.k + s];
    if ((uint32_t)row >= (uint32_t)t.R) continue;  // no expert
    f4 v = *(const f4*)(part + ((size_t)row * N4 + c) * 4);
    for (int p = 1; p < splits; ++p) v += *(const f4*)(part + (((size_t)p * t.R + row) * N4 + c) * 4);
    sum += v;
  }
  if (residual) {
    const uint2 raw = *(const uint2*)(residual + i * 4);
    sum += f4{half_lo(raw.x), half_hi(raw.x), half_lo(raw.y), half_hi(raw.y)};
  }
  uint2 o;
  o.x = half_bits(sum[0]) | (half_bits(sum[1]) << 16);
  o.y = half_bits(sum[2]) | (half_bits(sum[3]) << 16);
  *(uint2*)(y + i * 4) = o;
}

// One pair per workgroup: dh[r] = w U[r], dw = U[r] . h[r] + dy[m] . bias[e].
__global__ __launch_bounds__(kThreads) void share_grad_kernel(ExpertRouting t, const float* __restrict__ part,
                                                              int splits, const uint16_t* __restrict__ h,
                                                              const uint16_t* __restrict__ dy,
                                                              const uint16_t* __restrict__ bias,
                                                              uint16_t* __restrict__ dh, float* __restrict__ dweights,
                                                              int N, int d) {
  __shared__ float red[kThreads / 64];
  const int p = blockIdx.x, lane = threadIdx.x & 63;
  const int row = t.place[p], e = t.ids[p];
  if ((uint32_t)row >= (uint32_t)t.R || (uint32_t)e >= (uint32_t)t.E) {
    if (threadIdx.x == 0) dweights[p] = 0.0f;
    return;
  }
  const float w = t.weights[p];
  float dot = 0.0f;
  for (int c = threadIdx.x; c < d / 4; c += kThreads) {
    f4 u = *(const f4*)(part + (size_t)row * d + 4 * c);
    for (int q = 1; q < splits; ++q) u += *(const f4*)(part + ((size_t)q * t.R + row) * d + 4 * c);
    const uint2 raw = *(const uint2*)(h + (size_t)row * d + 4 * c);
    dot = __builtin_fmaf(u[0], half_lo(raw.x), dot);
    dot = __builtin_fmaf(u[1], half_hi(raw.x), dot);
    dot = __builtin_fmaf(u[2], half_lo(raw.y), dot);
    dot = __builtin_fmaf(u[3], half_hi(raw.y), dot);
    uint2 o;
    o.x = half_bits(u[0] * w) | (half_bits(u[1] * w) << 16);
    o.y = half_bits(u[2] * w) | (half_bits(u[3] * w) << 16);
    *(uint2*)(dh + (size_t)row * d + 4 * c) = o;
  }
  if (bias) {
    for (int c = threadIdx.x; c < N / 4; c += kThreads) {
      const uint2 a = *(const uint2*)(dy + (size_t)(p / t.k) * N + 4 * c);
      const uint2 b = *(const uint2*)(bias + (size_t)e * N + 4 * c);
      dot = __builtin_fmaf(half_lo(a.x), half_lo(b.x), dot);
      dot = __builtin_fmaf(half_hi(a.x), half_hi(b.x), dot);
      dot = __builtin_fmaf(half_lo(a.y), half_lo(b.y), dot);
      dot = __builtin_fmaf(half_hi(a.y), half_hi(b.y), dot);
    }
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) dot += __shfl_xor(dot, s);
  if (lane == 0) red[threadIdx.x >> 6] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = red[0];
    for (int i = 1; i < kThreads / 64; ++i) sum += red[i];
    dweights[p] = sum;
  }
}

// A wavefront per pair: its partial dots in order, and dy[m] . bias[e].
__global__ __launch_bounds__(kThreads) void dots_kernel(ExpertRouting t, const float* __restrict__ dots, int count,
                                                        const uint16_t* __restrict__ dy,
                                                        const uint16_t* __restrict__ bias,
                                                        float* __restrict__ dweights, int N) {
  const int p = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (p >= t.R) return;
  const int row = t.place[p], e = t.ids[p];
  float dot = 0.0f;
  if ((uint32_t)row < (uint32_t)t.R && (uint32_t)e < (uint32_t)t.E) {
    for (int i = lane; i < count; i += 64) dot += dots[(size_t)i * t.R + row];
    if (bias) {
      for (int c = lane; c < N / 4; c += 64) {
        const uint2 a = *(const uint2*)(dy + (size_t)(p / t.k) * N + 4 * c);
        const uint2 b = *(const uint2*)(bias + (size_t)e * N + 4 * c);
        dot = __builtin_fmaf(half_lo(a.x), half_lo(b.x), dot);
        dot = __builtin_fmaf(half_hi(a.x), half_hi(b.x), dot);
        dot = __builtin_fmaf(half_lo(a.y), half_lo(b.y), dot);
        dot = __builtin_fmaf(half_hi(a.y), half_hi(b.y), dot);
      }
    }
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) dot += __shfl_xor(dot, s);
  if (lane == 0) dweights[p] = dot;
}

}  // namespace

hipError_t launch_experts_dots(const ExpertRouting& t, const float* dots, int count, const uint16_t* dy,
                               const uint16_t* bias, float* dweights, int64_t N, hipStream_t stream) {
  const unsigned per = kThreads / 64;
  hipLaunchKernelGGL(dots_kernel, dim3(((unsigned)t.R + per - 1) / per), dim3(kThreads), 0, stream, t, dots, count, dy,
                     bias, dweights, (int)N);
  return hipGetLastError();
}

hipError_t launch_experts_sum(const ExpertRouting& t, const float* part, int splits, const uint16_t* residual,
                              uint16_t* y, int64_t N, hipStream_t stream) {
  const int64_t n = (int64_t)t.M * (N / 4);
  hipLaunchKernelGGL(sum_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, t, part,
                     splits, residual, y, (int)(N / 4));
  return hipGetLastError();
}

hipError_t launch_experts_share_grad(const ExpertRouting& t, const float* part, int splits, const uint16_t* h,
                                     const uint16_t* dy, const uint16_t* bias, uint16_t* dh, float* dweights,
                                     int64_t N, int64_t d, hipStream_t stream) {
  hipLaunchKernelGGL(share_grad_kernel, dim3((unsigned)t.R), dim3(kThreads), 0, stream, t, part, splits, h, dy, bias,
                     dh, dweights, (int)N, (int)d);
  return hipGetLastError();
}

}  // namespace paro
