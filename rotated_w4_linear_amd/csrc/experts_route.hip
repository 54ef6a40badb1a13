// gfx950 kernels of the experts' router:
//   p = softmax(l) over the E experts of a token, S its k largest logits (the
//   lower expert first where they are equal), w_s = p_s, or p_s / sum_S p;
// then the (token, slot) pairs in expert order, by counting: chunks of tokens
// count their pairs per expert, and each chunk then adds up the counts of the
// chunks before it and of the experts before each one, and places its pairs, in
// pair order inside an expert. Up to 128 tokens one launch does all of it. (A third
// kernel that turned the counts into first rows, one workgroup walking over the
// chunks: 16384 tokens, 8 of 256 experts, 234 us in all.)
//
// A wavefront takes a token. A lane has up to four neighbouring experts' logits,
// sorted, and the largest of the lanes' firsts is picked k times: the lowest lane
// that has it has the lowest expert. (More than 256 experts: a register for each
// 64 experts, and a ballot for each.) What bounds it: at a few tokens the launch
// and the k rounds, one after the other; at many the rounds' instructions (the
// logits are read once).
#include <algorithm>

#include "paro_internal.h"
#include "paro_types.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

// Tokens per chunk: few, so that the chunks fill the CUs, and more where there are
// so many chunks that adding up their counts would take longer: that work is the
// chunks' number squared, so that they stay at 1024 or fewer for as long as a chunk
// has at most 4096 pairs (its tables fill the LDS), and at 4096 in all. (Given ids of
// 2^20 tokens, chunks of 256 | these: 2 of 256 experts 687 | 72 us, 1 of 1024 2929 |
// 217, 8 of 60 225 | 114.)
constexpr int kOneChunk = 128, kChunkPairs = 4096;
int chunk_tokens(int64_t M, int k) {
  if (M <= kOneChunk) return kOneChunk;
  int n = M <= 16384 ? 64 : M <= 32768 ? 128 : 256;
  while (M > 1024 * (int64_t)n && 2 * n * k <= kChunkPairs) n *= 2;
  return n;
}
// Counts of a chunk: whole words of two
__host__ __device__ __forceinline__ int count_stride(int E) { return (E + 2) & ~1; }
constexpr int kThreads = 1024, kWaves = kThreads / 64;

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
  auto with = [&](int moved) { v += __builtin_bit_cast(float, moved); };
  with(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x111, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x112, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x114, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x118, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xa, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x143, 0xc, 0xf, false));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// e^x, x <= 0: an argument rounded once, an ulp or two of exp2; 0 below 2^-126
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(1.4426950408889634f * x); }

// Largest of the lanes' numbers, in every lane (rows of 16 by shifts, then across
// them: a few cycles a step, where a shuffle through LDS takes a hundred).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto with = [&](int moved) { v = max(v, (uint32_t)moved); };
  with(__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));  // row_shr 1
  with(__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));  // row_shr 2
  with(__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));  // row_shr 4
  with(__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));  // row_shr 8
  with(__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));  // row_bcast 15
  with(__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));  // row_bcast 31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The k largest of a token's E logits: lane s < k returns the s-th's expert (-1:
// none left) and its weight. EPL: logits per lane, neighbours up to four (then a
// lane's are sorted first), 64 apart beyond.
template <class T, int EPL>
__device__ __forceinline__ void route_token(const typename T::raw* __restrict__ l, int E, int k, int normalize,
                                            int lane, int& id, float& weight) {
  constexpr bool kSorted = EPL <= 4;
  uint32_t r[EPL], all[EPL];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = kSorted ? EPL * lane + j : 64 * j + lane;
    const float v = e < E ? T::value(l[e]) : -__builtin_inff();
    bad = bad || v != v;
    all[j] = r[j] = rank_of(v);
  }
  int at[EPL];  // which of the lane's logits
  if constexpr (kSorted) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) at[j] = j;
    // (neighbours change places only where the later one is larger: equal ones stay in order)
#pragma unroll
    for (int n = EPL - 1; n > 0; --n)
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const bool swap = r[j + 1] > r[j];
        const uint32_t a = r[j], b = r[j + 1];
        const int x = at[j], y = at[j + 1];
        r[j] = swap ? b : a;
        r[j + 1] = swap ? a : b;
        at[j] = swap ? y : x;
        at[j + 1] = swap ? x : y;
      }
  }
  uint32_t mine = 0;  // lane s: the s-th logit's rank
  id = -1;
  uint32_t high = 0;
  for (int s = 0; s < k; ++s) {
    uint32_t best = r[0];
    if constexpr (!kSorted) {
#pragma unroll
      for (int j = 1; j < EPL; ++j) best = max(best, r[j]);
    }
    best = wave_max(best);
    if (best == 0) break;
    if (s == 0) high = best;
    int expert = 0;
    if constexpr (kSorted) {
      const int from = __builtin_ctzll(__ballot(r[0] == best));
      expert = EPL * from + __builtin_amdgcn_readlane(at[0], from);
      const bool taken = lane == from;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        r[j] = taken ? (j + 1 < EPL ? r[j + 1 < EPL ? j + 1 : j] : 0u) : r[j];
        if (j + 1 < EPL) at[j] = taken ? at[j + 1] : at[j];
      }
    } else {
      bool found = false;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const uint64_t has = __ballot(r[j] == best);
        if (!found && has != 0) {
          found = true;
          const int from = __builtin_ctzll(has);
          expert = 64 * j + from;
          if (lane == from) r[j] = 0;
        }
      }
    }
    if (lane == s) {
      mine = best;
      id = expert;
    }
  }
  const float top = value_of(high);
  const float e = id >= 0 ? fast_exp(value_of(mine) - top) : 0.0f;
  float total = e;
  if (!normalize) {
    total = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) total += all[j] ? fast_exp(value_of(all[j]) - top) : 0.0f;
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

// LDS of a chunk: its pairs' experts (those without one: bucket E), for each
// batch of 64 pairs the rows of every bucket before it in the chunk, and each
// bucket's first row.
struct ChunkLds {
  int* ids;       // [pairs]
  int* first;     // [E + 1]
  int* red;       // [kWaves]
  uint16_t* pre;  // [batches][E + 1]
};
__device__ __forceinline__ ChunkLds chunk_lds(uint8_t* at, int pairs, int E) {
  ChunkLds l;
  l.ids = (int*)at;
  l.first = l.ids + pairs;
  l.red = l.first + E + 1;
  l.pre = (uint16_t*)(l.red + kWaves);
  return l;
}
size_t chunk_lds_bytes(int64_t pairs, int E) {
  return (size_t)(pairs + E + 1 + kWaves) * 4 + (size_t)((pairs + 63) / 64) * (E + 1) * 2;
}

// Places a chunk's pairs behind the rows that first holds: a row is first[e], the
// expert's pairs in the batches before, and those before it in its batch. order
// has -1 in the rows of bucket E.
__device__ __forceinline__ void place_chunk(const ChunkLds& l, int pairs, int pair0, int E, int* __restrict__ order,
                                            int* __restrict__ place) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int batches = (pairs + 63) >> 6, EB = E + 1;
  for (int i = tid; i < batches * EB; i += kThreads) l.pre[i] = 0;
  __syncthreads();
  auto batch = [&](int b, bool& in, uint32_t& e, uint64_t& m) {
    const int p = 64 * b + lane;
    in = p < pairs;
    e = in ? (uint32_t)l.ids[p] : 2047u;  // (lanes past the end: a bucket of their own)
    m = same_lanes(e);
  };
  bool in;
  uint32_t e;
  uint64_t m;
  for (int b = w; b < batches; b += kWaves) {
    batch(b, in, e, m);
    if (in && (m & ((uint64_t(1) << lane) - 1)) == 0) l.pre[b * EB + e] = (uint16_t)__popcll(m);
  }
  __syncthreads();
  if (batches > 1) {
    for (int x = tid; x < EB; x += kThreads) {
      int at = 0;
      for (int b = 0; b < batches; ++b) {
        const int n = l.pre[b * EB + x];
        l.pre[b * EB + x] = (uint16_t)at;
        at += n;
      }
    }
    __syncthreads();
  }
  for (int b = w; b < batches; b += kWaves) {
    batch(b, in, e, m);
    if (in) {
      const int before = batches > 1 ? l.pre[b * EB + e] : 0;
      const int row = l.first[e] + before + __popcll(m & ((uint64_t(1) << lane) - 1));
      const bool live = e < (uint32_t)E;
      order[row] = live ? pair0 + 64 * b + lane : -1;
      place[pair0 + 64 * b + lane] = live ? row : -1;
    }
  }
}

// first[e], e's pairs, to the first row of e: the rows of the experts before it
// (and offsets, if given; offsets[E] is that of bucket E). more[e] is added.
template <class More>
__device__ __forceinline__ void scan_first(const ChunkLds& l, int E, int* offsets, More more) {
  int carry = 0;
  for (int e0 = 0; e0 < E + 1; e0 += kThreads) {
    const int e = e0 + (int)threadIdx.x;
    int total;
    const int at = carry + block_scan(e <= E ? l.first[e] : 0, l.red, &total);
    if (e <= E) {
      if (offsets) offsets[e] = at;
      l.first[e] = at + more(e);
    }
    carry += total;
  }
  __syncthreads();
}

__device__ __forceinline__ int bucket(int id, int E) { return (uint32_t)id < (uint32_t)E ? id : E; }

// The router (ROUTE), or given ids, of one chunk of tokens, and its counts. With
// one chunk in all (gridDim.x == 1) also the offsets and the tables.
template <class T, int EPL, bool ROUTE>
__global__ __launch_bounds__(kThreads) void route_kernel(const typename T::raw* __restrict__ logits,
                                                         const int* given, int M, int E, int k, int chunk,
                                                         int normalize, int* ids, float* __restrict__ weights,
                                                         uint16_t* __restrict__ counts, int* __restrict__ offsets,
                                                         int* __restrict__ order, int* __restrict__ place) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int t0 = chunk * blockIdx.x, tokens = min(chunk, M - t0);
  const int pairs = tokens * k;
  const ChunkLds l = chunk_lds(dyn, min(chunk, M) * k, E);
  for (int i = tid; i <= E; i += kThreads) l.first[i] = 0;
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
        l.ids[t * k + lane] = bucket(id, E);
        atomicAdd(&l.first[bucket(id, E)], 1);
      }
    }
  } else {
    for (int p = tid; p < pairs; p += kThreads) {
      const int e = bucket(given[(size_t)t0 * k + p], E);
      l.ids[p] = e;
      atomicAdd(&l.first[e], 1);
    }
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (int i = tid; i < count_stride(E); i += kThreads)
      counts[(size_t)blockIdx.x * count_stride(E) + i] = (uint16_t)(i <= E ? l.first[i] : 0);
    return;
  }
  scan_first(l, E, offsets, [](int) { return 0; });
  place_chunk(l, pairs, 0, E, order, place);
}

// The tables of one chunk, from all chunks' counts, two buckets a word. (Every
// workgroup reads them all: 132 KB at 16384 tokens and 256 experts, from L2.)
__global__ __launch_bounds__(kThreads) void place_kernel(const int* __restrict__ ids, int M, int E, int k, int chunk,
                                                         const uint32_t* __restrict__ counts, int chunks,
                                                         int* __restrict__ offsets, int* __restrict__ order,
                                                         int* __restrict__ place) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ int before[kExpertsMax + 1];
  const int tid = threadIdx.x, mine = blockIdx.x;
  const int t0 = chunk * mine, pairs = min(chunk, M - t0) * k;
  const int pair0 = t0 * k;
  const ChunkLds l = chunk_lds(dyn, chunk * k, E);
  for (int i = tid; i <= E; i += kThreads) l.first[i] = before[i] = 0;
  __syncthreads();
  for (int p = tid; p < pairs; p += kThreads) l.ids[p] = bucket(ids[pair0 + p], E);
  // parts of the chunks side by side, as many as there are threads for
  const int words = count_stride(E) / 2, parts = kThreads / words, part = tid / words, i = tid - part * words;
  if (part < parts) {
    int sum0 = 0, sum1 = 0, all0 = 0, all1 = 0;
#pragma unroll 8
    for (int c = part; c < chunks; c += parts) {
      const uint32_t n = counts[(size_t)c * words + i];
      const int n0 = (int)(n & 0xffffu), n1 = (int)(n >> 16);
      all0 += n0;
      all1 += n1;
      sum0 += c < mine ? n0 : 0;
      sum1 += c < mine ? n1 : 0;
    }
    // (whole numbers: the same in any order)
    atomicAdd(&l.first[2 * i], all0);
    atomicAdd(&before[2 * i], sum0);
    if (2 * i + 1 <= E) {
      atomicAdd(&l.first[2 * i + 1], all1);
      atomicAdd(&before[2 * i + 1], sum1);
    }
  }
  __syncthreads();
  scan_first(l, E, mine == 0 ? offsets : nullptr, [&](int e) { return before[e]; });
  place_chunk(l, pairs, pair0, E, order, place);
}

// Gradient at the logits, a wavefront per token. Normalised weights:
//   dl_i = w_i (dw_i - sum_S w dw) for i in S, else 0;
// p itself: dl_j = [j in S] p_j dw_j - p_j sum_S p dw, NaN at every expert where a
// logit is NaN or +inf, and 0 for a token without an expert.
template <class T>
__global__ __launch_bounds__(256) void route_backward_kernel(const typename T::raw* __restrict__ logits,
                                                                  const int* __restrict__ ids,
                                                                  const float* __restrict__ weights,
                                                                  const float* __restrict__ dweights, int M, int E,
                                                                  int k, int normalize,
                                                                  typename T::raw* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63, m = blockIdx.x * 4 + (threadIdx.x >> 6);
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
    for (int e = lane; e < E; e += 64) {
      const float x = T::value(l[e]);
      total += x == -__builtin_inff() ? 0.0f : expf(x - top);
    }
    total = wave_sum(total);
  }
  const bool any = __ballot(id >= 0) != 0 && total != 0.0f;  // (a NaN is not 0)
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    float v = 0.0f;
    if (!normalize && e < E && any) v = -(expf(T::value(l[e]) - top) / total) * inner;
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

// (dynamic LDS beyond what a launch takes by itself)
template <class K>
hipError_t allow_lds(K kernel, size_t bytes) {
  if (bytes <= 65536) return hipSuccess;
  return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <class T, bool ROUTE>
hipError_t launch_route(int chunk, int chunks, hipStream_t stream, const void* logits, const int* given, int M, int E,
                        int k, int normalize, int* ids, float* weights, uint16_t* counts, int* offsets, int* order,
                        int* place) {
  const size_t lds = chunk_lds_bytes((int64_t)std::min(chunk, M) * k, E);
  auto go = [&](auto kernel) {
    const hipError_t e = allow_lds(kernel, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)chunks), dim3(kThreads), (unsigned)lds, stream,
                       (const typename T::raw*)logits, given, M, E, k, chunk, normalize, ids, weights, counts, offsets,
                       order, place);
    return hipGetLastError();
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

size_t experts_route_scratch(int64_t M, int E, int k) {
  const int64_t chunk = chunk_tokens(M, k), chunks = (M + chunk - 1) / chunk;
  return chunks > 1 ? (size_t)chunks * count_stride(E) * 2 : 0;
}

hipError_t launch_experts_route(const void* logits, int type, int64_t M, int E, int k, int normalize, int* ids,
                                float* weights, int* offsets, int* order, int* place, void* scratch,
                                hipStream_t stream) {
  const int chunk = chunk_tokens(M, k), chunks = (int)((M + chunk - 1) / chunk);
  uint16_t* counts = (uint16_t*)scratch;
  hipError_t e = hipSuccess;
  if (!logits)
    e = launch_route<F32, false>(chunk, chunks, stream, nullptr, ids, (int)M, E, k, 0, nullptr, nullptr, counts,
                                 offsets, order, place);
  else
    with_type(type, [&](auto t) {
      e = launch_route<decltype(t), true>(chunk, chunks, stream, logits, nullptr, (int)M, E, k, normalize, ids,
                                          weights, counts, offsets, order, place);
    });
  if (e != hipSuccess || chunks == 1) return e;
  const size_t lds = chunk_lds_bytes((int64_t)chunk * k, E);
  if ((e = allow_lds(place_kernel, lds)) != hipSuccess) return e;
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)chunks), dim3(kThreads), (unsigned)lds, stream, ids, (int)M, E, k,
                     chunk, (const uint32_t*)scratch, chunks, offsets, order, place);
  return hipGetLastError();
}

hipError_t launch_experts_route_backward(const void* logits, int type, int64_t M, int E, int k, int normalize,
                                         const int* ids, const float* weights, const float* dweights, void* dlogits,
                                         hipStream_t stream) {
  const unsigned blocks = (unsigned)((M + 3) / 4);
  with_type(type, [&](auto t) {
    typedef decltype(t) T;
    hipLaunchKernelGGL(route_backward_kernel<T>, dim3(blocks), dim3(256), 0, stream,
                       (const typename T::raw*)logits, ids, weights, dweights, (int)M, E, k, normalize,
                       (typename T::raw*)dlogits);
  });
  return hipGetLastError();
}

}  // namespace paro
