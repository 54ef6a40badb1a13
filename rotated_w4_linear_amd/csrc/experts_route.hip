// gfx950 kernels of the experts' router:
//   p = softmax(l) over the E experts of a token, S its k largest logits (the
//   lower expert first where they are equal), w_s = p_s, or p_s / sum_S p;
// then the (token, slot) pairs in expert order, by counting: chunks of 64
// tokens count their pairs per expert, one workgroup turns the counts into each
// chunk's first row of every expert, and the chunks place their pairs, in pair
// order inside an expert. Up to 64 tokens one workgroup does all of it in one
// launch.
//
// A wavefront takes a token, 64 experts at a time in a register per lane, and
// picks the largest of (logit, -expert) k times with a reduction over the
// lanes. What bounds it: at a few tokens the launch and the k reductions one
// after the other; at many their instructions (the logits are read once).
#include "paro_internal.h"
#include "paro_types.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

constexpr int kChunkTokens = 64;
constexpr int kThreads = 256, kWaves = kThreads / 64;

// Order of the floats as unsigned numbers, never 0 for an expert that can be
// taken; -inf and NaN: 0.
__device__ __forceinline__ uint32_t rank_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);  // (-0 is 0)
  if (!(v > -__builtin_inff())) return 0u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t r) {
  return __builtin_bit_cast(float, r & 0x80000000u ? r & 0x7fffffffu : ~r);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

// The k largest of a token's E logits: lane s < k returns the s-th's expert (-1:
// none left) and its weight.
template <class T, int EPL>
__device__ __forceinline__ void route_token(const typename T::raw* __restrict__ l, int E, int k, int normalize,
                                            int lane, int& id, float& weight) {
  uint32_t r[EPL];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = 64 * j + lane;
    const float v = e < E ? T::value(l[e]) : -__builtin_inff();
    bad = bad || v != v;
    r[j] = rank_of(v);
  }
  uint32_t all[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) all[j] = r[j];
  uint32_t mine = 0;  // lane s: the s-th logit's rank
  id = -1;
  uint32_t high = 0;
  for (int s = 0; s < k; ++s) {
    uint32_t best = 0, expert = ~0u;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (r[j] > best) {  // (the lower expert stays where they are equal)
        best = r[j];
        expert = 64 * j + lane;
      }
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) {
      const uint32_t ob = __shfl_xor(best, x), oe = __shfl_xor(expert, x);
      if (ob > best || (ob == best && oe < expert)) {
        best = ob;
        expert = oe;
      }
    }
    if (best == 0) break;
    if (s == 0) high = best;
    if (lane == s) {
      mine = best;
      id = (int)expert;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (expert == (uint32_t)(64 * j + lane)) r[j] = 0;
  }
  const float top = value_of(high);
  const float e = id >= 0 ? expf(value_of(mine) - top) : 0.0f;
  float total = e;
  if (!normalize) {
    total = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (all[j]) total += expf(value_of(all[j]) - top);
  }
  total = wave_sum(total);
  weight = id >= 0 ? e / total : 0.0f;
  // a NaN among the logits shows in the token's weights
  if (__ballot(bad) != 0 && id >= 0) weight = __builtin_nanf("");
}

// Lanes of this wavefront with the same number, of at most 11 bits.
__device__ __forceinline__ uint64_t same_lanes(uint32_t v) {
  uint64_t m = ~uint64_t(0);
#pragma unroll
  for (int b = 0; b < 11; ++b) {
    const uint64_t set = __ballot((v >> b) & 1u);
    m &= (v >> b) & 1u ? set : ~set;
  }
  return m;
}

// Exclusive scan over the workgroup's threads; red: kWaves words of LDS.
__device__ __forceinline__ int block_scan(int v, int* red, int* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const int o = __shfl_up(s, x);
    if (lane >= x) s += o;
  }
  __syncthreads();
  if (lane == 63) red[w] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    before += i < w ? red[i] : 0;
    all += red[i];
  }
  *total = all;
  return before + s - v;
}

// Places a chunk's pairs (ids in LDS, -1 and others outside [0, E): bucket E).
// pre[b][e] becomes the first row of batch b's (64 pairs) pairs of expert e:
// base(e) for batch 0. order has -1 in the rows of bucket E.
template <class Base>
__device__ __forceinline__ void place_chunk(const int* ids, int pairs, int pair0, int E, int* pre, Base base,
                                            int* __restrict__ order, int* __restrict__ place) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int batches = (pairs + 63) >> 6, EB = E + 1;
  for (int i = tid; i < batches * EB; i += kThreads) pre[i] = 0;
  __syncthreads();
  for (int b = w; b < batches; b += kWaves) {
    const int p = 64 * b + lane;
    const bool in = p < pairs;
    const uint32_t e = in ? (uint32_t)ids[p] : 2047u;  // (lanes past the end: a bucket of their own)
    const uint64_t m = same_lanes(e);
    if (in && (m & ((uint64_t(1) << lane) - 1)) == 0) pre[b * EB + e] = __popcll(m);
  }
  __syncthreads();
  for (int e = tid; e < EB; e += kThreads) {
    int at = base(e);
    for (int b = 0; b < batches; ++b) {
      const int n = pre[b * EB + e];
      pre[b * EB + e] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int b = w; b < batches; b += kWaves) {
    const int p = 64 * b + lane;
    const bool in = p < pairs;
    const uint32_t e = in ? (uint32_t)ids[p] : 2047u;
    const uint64_t m = same_lanes(e);
    if (in) {
      const int row = pre[b * EB + e] + __popcll(m & ((uint64_t(1) << lane) - 1));
      const bool live = e < (uint32_t)E;
      order[row] = live ? pair0 + p : -1;
      place[pair0 + p] = live ? row : -1;
    }
  }
}

__device__ __forceinline__ int bucket(int id, int E) { return (uint32_t)id < (uint32_t)E ? id : E; }

// The router (ROUTE), or given ids, of one chunk of tokens, and its counts. With
// one chunk in all (gridDim.x == 1) also the offsets and the tables.
template <class T, int EPL, bool ROUTE>
__global__ __launch_bounds__(kThreads) void route_kernel(const typename T::raw* __restrict__ logits,
                                                         const int* given, int M, int E, int k, int normalize,
                                                         int* ids, float* __restrict__ weights,
                                                         int* __restrict__ counts, int* __restrict__ offsets,
                                                         int* __restrict__ order, int* __restrict__ place) {
  __shared__ int lids[kChunkTokens * kExpertsMaxK];
  __shared__ int hist[kExpertsMax + 1];
  __shared__ int red[kWaves];
  extern __shared__ int pre[];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int t0 = kChunkTokens * blockIdx.x, tokens = min(kChunkTokens, M - t0);
  const int pairs = tokens * k, EB = E + 1;
  for (int i = tid; i < EB; i += kThreads) hist[i] = 0;
  __syncthreads();
  if constexpr (ROUTE) {
    for (int t = w; t < tokens; t += kWaves) {
      int id;
      float weight;
      route_token<T, EPL>(logits + (size_t)(t0 + t) * E, E, k, normalize, lane, id, weight);
      if (lane < k) {
        const size_t p = (size_t)(t0 + t) * k + lane;
        ids[p] = id;
        weights[p] = weight;
        lids[t * k + lane] = bucket(id, E);
        atomicAdd(&hist[bucket(id, E)], 1);
      }
    }
  } else {
    for (int p = tid; p < pairs; p += kThreads) {
      const int e = bucket(given[(size_t)t0 * k + p], E);
      lids[p] = e;
      atomicAdd(&hist[e], 1);
    }
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (int i = tid; i < EB; i += kThreads) counts[(size_t)blockIdx.x * EB + i] = hist[i];
    return;
  }
  int carry = 0;
  for (int e0 = 0; e0 < EB; e0 += kThreads) {
    const int e = e0 + tid, n = e < EB ? hist[e] : 0;
    int total;
    const int at = carry + block_scan(n, red, &total);
    if (e < EB) {
      offsets[e] = at;  // (offsets[E]: the first row of bucket E, the pairs without an expert)
      hist[e] = at;
    }
    carry += total;
  }
  __syncthreads();
  place_chunk(lids, pairs, 0, E, pre, [&](int e) { return hist[e]; }, order, place);
}

// counts [chunks][E + 1] to each chunk's first row of every expert, and the offsets
__global__ __launch_bounds__(kThreads) void scan_kernel(int* counts, int chunks, int E, int* __restrict__ offsets) {
  __shared__ int red[kWaves];
  const int EB = E + 1;
  int carry = 0;
  for (int e0 = 0; e0 < EB; e0 += kThreads) {
    const int e = e0 + (int)threadIdx.x;
    int n = 0;
    if (e < EB)
      for (int c = 0; c < chunks; ++c) n += counts[(size_t)c * EB + e];
    int total;
    int at = carry + block_scan(n, red, &total);
    if (e < EB) {
      offsets[e] = at;
      for (int c = 0; c < chunks; ++c) {
        const int m = counts[(size_t)c * EB + e];
        counts[(size_t)c * EB + e] = at;
        at += m;
      }
    }
    carry += total;
  }
}

__global__ __launch_bounds__(kThreads) void place_kernel(const int* __restrict__ ids, int M, int E, int k,
                                                         const int* __restrict__ base, int* __restrict__ order,
                                                         int* __restrict__ place) {
  __shared__ int lids[kChunkTokens * kExpertsMaxK];
  extern __shared__ int pre[];
  const int t0 = kChunkTokens * blockIdx.x, pairs = min(kChunkTokens, M - t0) * k;
  const int pair0 = t0 * k;
  for (int p = threadIdx.x; p < pairs; p += kThreads) lids[p] = bucket(ids[pair0 + p], E);
  __syncthreads();
  const int* mine = base + (size_t)blockIdx.x * (E + 1);
  place_chunk(lids, pairs, pair0, E, pre, [&](int e) { return mine[e]; }, order, place);
}

// Gradient at the logits, a wavefront per token. Normalised weights:
//   dl_i = w_i (dw_i - sum_S w dw) for i in S, else 0;
// p itself: dl_j = [j in S] p_j dw_j - p_j sum_S p dw.
template <class T>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const typename T::raw* __restrict__ logits,
                                                                  const int* __restrict__ ids,
                                                                  const float* __restrict__ weights,
                                                                  const float* __restrict__ dweights, int M, int E,
                                                                  int k, int normalize,
                                                                  typename T::raw* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63, m = blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (m >= M) return;
  int id = -1;
  float w = 0.0f, dw = 0.0f;
  if (lane < k) {
    id = bucket(ids[(size_t)m * k + lane], E);
    if (id == E) id = -1;
    if (id >= 0) {
      w = weights[(size_t)m * k + lane];
      dw = dweights[(size_t)m * k + lane];
    }
  }
  const float inner = wave_sum(w * dw);
  const float taken = normalize ? w * (dw - inner) : w * dw;
  const typename T::raw* l = logits + (size_t)m * E;
  float top = -__builtin_inff(), total = 0.0f;
  if (!normalize) {
    for (int e = lane; e < E; e += 64) top = fmaxf(top, T::value(l[e]));
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    for (int e = lane; e < E; e += 64) total += top > -__builtin_inff() ? expf(T::value(l[e]) - top) : 0.0f;
    total = wave_sum(total);
  }
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    float v = 0.0f;
    if (!normalize && e < E && total > 0.0f) v = -(expf(T::value(l[e]) - top) / total) * inner;
    for (int s = 0; s < k; ++s) {
      const int i = __shfl(id, s);
      const float t = __shfl(taken, s);
      if (i == e) v += t;
    }
    if (e < E) dlogits[(size_t)m * E + e] = T::pack(v);
  }
}

int experts_per_lane(int E) {
  int n = 1;
  while (64 * n < E) n *= 2;
  return n;
}
unsigned place_lds(int64_t tokens, int E, int k) { return (unsigned)((tokens * k + 63) / 64 * (E + 1) * 4); }

template <class T, bool ROUTE>
void launch_route(int chunks, unsigned lds, hipStream_t stream, const void* logits, const int* given, int M, int E,
                  int k, int normalize, int* ids, float* weights, int* counts, int* offsets, int* order, int* place) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)chunks), dim3(kThreads), lds, stream, (const typename T::raw*)logits,
                       given, M, E, k, normalize, ids, weights, counts, offsets, order, place);
  };
  switch (ROUTE ? experts_per_lane(E) : 1) {
    case 1: return go(route_kernel<T, 1, ROUTE>);
    case 2: return go(route_kernel<T, 2, ROUTE>);
    case 4: return go(route_kernel<T, 4, ROUTE>);
    case 8: return go(route_kernel<T, 8, ROUTE>);
    default: return go(route_kernel<T, 16, ROUTE>);
  }
}

}  // namespace

size_t experts_route_scratch(int64_t M, int E) {
  const int64_t chunks = (M + kChunkTokens - 1) / kChunkTokens;
  return chunks > 1 ? (size_t)chunks * (E + 1) * 4 : 0;
}

hipError_t launch_experts_route(const void* logits, int type, int64_t M, int E, int k, int normalize, int* ids,
                                float* weights, int* offsets, int* order, int* place, void* scratch,
                                hipStream_t stream) {
  const int chunks = (int)((M + kChunkTokens - 1) / kChunkTokens);
  const unsigned lds = chunks == 1 ? place_lds(M, E, k) : 0;
  int* counts = (int*)scratch;
  if (!logits)
    launch_route<F32, false>(chunks, lds, stream, nullptr, ids, (int)M, E, k, 0, nullptr, nullptr, counts, offsets,
                             order, place);
  else
    with_type(type, [&](auto t) {
      launch_route<decltype(t), true>(chunks, lds, stream, logits, nullptr, (int)M, E, k, normalize, ids, weights,
                                      counts, offsets, order, place);
    });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks == 1) return e;
  hipLaunchKernelGGL(scan_kernel, dim3(1), dim3(kThreads), 0, stream, counts, chunks, E, offsets);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)chunks), dim3(kThreads), place_lds(kChunkTokens, E, k), stream, ids,
                     (int)M, E, k, counts, order, place);
  return hipGetLastError();
}

hipError_t launch_experts_route_backward(const void* logits, int type, int64_t M, int E, int k, int normalize,
                                         const int* ids, const float* weights, const float* dweights, void* dlogits,
                                         hipStream_t stream) {
  const unsigned blocks = (unsigned)((M + kWaves - 1) / kWaves);
  with_type(type, [&](auto t) {
    typedef decltype(t) T;
    hipLaunchKernelGGL(route_backward_kernel<T>, dim3(blocks), dim3(kThreads), 0, stream,
                       (const typename T::raw*)logits, ids, weights, dweights, (int)M, E, k, normalize,
                       (typename T::raw*)dlogits);
  });
  return hipGetLastError();
}

}  // namespace paro
