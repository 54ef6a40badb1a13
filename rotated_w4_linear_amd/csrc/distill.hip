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
// the rest is a class of its own); the entries are done in fp64 by one
// wavefront, and the sum of everything is the rest's plus the entries': where
// teacher and student agree, L is a small difference, and an error of the rest's
// sum then enters by Q - P only. The rest has a maximum of its own: below the
// entries' by 88 T its exponentials would all be 0, and the loss infinite. A second
// pass reads z again, from the memory-side cache, and writes the gradient.
//
// What bounds it: with a gradient memory (4096 rows of 131072 bf16 in 476 us, 4.5 TB/s
// of one read and one write, the second read in part from the cache; 8% longer with
// stores that go through it); on short rows the entries' chain of latencies, 8 us,
// which the other workgroups of the CU cover. (In an earlier form, 650 us: reductions
// over the whole workgroup for the entries too, 14 us a row; rows kept in registers
// between the passes, 1024 lanes a row, 706 us, nothing then covers the chain.)
#include "paro_internal.h"
#include "paro_types.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
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

// Reductions over a wavefront in a fixed order, in every lane: rows of 16 lanes by
// shifts, then across them, then the last lane's. `none` takes no part.
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float v, float none) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),
                                                               __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v, double none) {
  const uint64_t a = __builtin_bit_cast(uint64_t, v), b = __builtin_bit_cast(uint64_t, none);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)b, (int)a, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(b >> 32), (int)(a >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float last_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t a = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)a, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(a >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <class V, class Op>
__device__ __forceinline__ V wave_reduce(V v, V none, Op op) {
  v = op(v, moved<0x111, 0xf>(v, none));
  v = op(v, moved<0x112, 0xf>(v, none));
  v = op(v, moved<0x114, 0xf>(v, none));
  v = op(v, moved<0x118, 0xf>(v, none));
  v = op(v, moved<0x142, 0xa>(v, none));
  v = op(v, moved<0x143, 0xc>(v, none));
  return last_lane(v);
}
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
  return wave_reduce(v, (V)0, [](V a, V b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, -kInf, [](float a, float b) { return fmaxf(a, b); });
}

// The teacher's value i, of any type (the same for all lanes).
__device__ __forceinline__ float value_of(const void* p, int type, int64_t i) {
  if (type == PARO_TYPE_F32) return ((const float*)p)[i];
  const uint16_t raw = ((const uint16_t*)p)[i];
  return type == PARO_TYPE_F16 ? F16::value(raw) : BF16::value(raw);
}

template <class Z, int NT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(8))) void distill_kernel(DistillArgs a, int value_type) {
  typedef typename Z::raw raw;
  constexpr int VE = Vec<Z>::VE, NW = NT / 64, B = 2;
  __shared__ float wmax[NW], wsum[NW];
  __shared__ float factor;
  __shared__ int none_left;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63, V = a.V, K = a.K;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the wavefront that does the entries: another one in the workgroups of a CU, which
  // would all keep the same SIMD busy
  const int own = (int)(blockIdx.x + (blockIdx.x >> 8)) & (NW - 1);
  double* p = (double*)dyn;                   // [K] the entries' masses, then their gradients
  double* e = p + K;                          // [K] e^(z / T) in the sum's unit
  float* zj = (float*)(e + K);                // [K] the student there
  int* index = (int*)(zj + K);                // [K] -1: no entry
  uint32_t* bits = (uint32_t*)(index + K);    // V bits and VE
  const int64_t m = blockIdx.x;
  const raw* z = (const raw*)a.z + m * V;
  raw* dz = a.dz ? (raw*)a.dz + m * V : nullptr;
  const float weight = a.weight ? a.weight[m] : 1.0f;
  const bool rest = a.lse != nullptr;
  // the first 64 entries and lse, on their way while the bitmap is cleared
  int j0 = -1;
  float t0 = -kInf, z0 = 0.0f, lse = 0.0f;
  if (w == own) {
    if (lane < K) {
      j0 = a.index[m * K + lane];
      t0 = value_of(a.values, value_type, m * K + lane);
    }
    if (rest) lse = a.lse[m];
    if ((uint32_t)j0 < (uint32_t)V) z0 = Z::value(z[j0]);
  }
  // 16-byte vectors from the first aligned element on; the elements before and
  // behind them one by one. Element j has bit j + skip: a vector's lie in one byte.
  const int head = min(V, (int)((16 - ((uintptr_t)z & 15)) & 15) / (int)sizeof(raw));
  const int nvec = (V - head) / VE, tail0 = head + nvec * VE, skip = (VE - head % VE) % VE;
  const int vbase = (head + skip) / VE;  // the first vector, in units of VE bits

  auto zeros = [&]() {
    if (dz) {
      for (int j = tid; j < head; j += NT) dz[j] = (raw)0;
      for (int v = tid; v < nvec; v += NT) *(u4*)(dz + head + v * VE) = u4{0u, 0u, 0u, 0u};
      for (int j = tail0 + tid; j < V; j += NT) dz[j] = (raw)0;
    }
    if (tid == 0) a.loss[m] = 0.0f;
  };
  if (weight == 0.0f) return zeros();  // (a row that is left out: whatever it holds)

  // the teacher's entries
  const double it = 1.0 / (double)a.temperature;
  const int words = (V + VE + 31) / 32;
  for (int i = tid; i < words; i += NT) bits[i] = 0;
  __syncthreads();
  double psum = 0.0, pscale = 1.0, P = 0.0, A = 1.0;
  float zmax = -kInf;  // the student's largest at the entries
  bool twice = false;
  if (w == own) {
    float tmax = -kInf;
    bool again = false, entries = false;
#pragma unroll 1
    for (int i = lane; i < K; i += 64) {
      const int j = i < 64 ? j0 : a.index[m * K + i];
      const bool in = (uint32_t)j < (uint32_t)V;
      const float t = i < 64 ? t0 : value_of(a.values, value_type, m * K + i);
      index[i] = in ? j : -1;
      p[i] = (double)t * it;
      if (!in) continue;
      const float x = i < 64 ? z0 : Z::value(z[j]);
      zj[i] = x;
      zmax = fmaxf(zmax, x);
      entries = entries || t > -kInf || t != t;
      tmax = fmaxf(tmax, t);
      const uint32_t b = 1u << ((j + skip) & 31);
      again = again || (atomicOr(&bits[(j + skip) >> 5], b) & b) != 0;
    }
    twice = __ballot(again) != 0;
    const bool any = __ballot(entries) != 0;
    if (lane == 0) none_left = !rest && !any;  // (a mask that leaves nothing of the teacher)
    psum = tmax;
  }
  __syncthreads();
  if (w == own) {  // (the others go on meanwhile)
    const double ref = rest ? (double)lse : (double)wave_max((float)psum) * it;
    psum = 0.0;
#pragma unroll 1
    for (int i = lane; i < K; i += 64) {
      const double v = index[i] >= 0 ? exp(p[i] - ref) : 0.0;
      p[i] = v;
      psum += v;
    }
    psum = wave_sum(psum);
    if (rest) {
      P = fmax(1.0 - psum, 0.0);
      A = psum + P;
    } else {
      pscale = 1.0 / psum;
    }
  }

  // all vectors of the lane, the next two on their way meanwhile (dz may be z: a
  // lane reads a vector before anyone writes it)
  auto stream = [&](auto use) {
    const u4* src = (const u4*)(z + head);
    u4 now[B], next[B];
    auto load = [&](int v0, u4* to) {
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (v0 + b * NT < nvec) to[b] = src[v0 + b * NT];
    };
    load(tid, now);
    for (int v0 = tid; v0 < nvec; v0 += B * NT) {
      load(v0 + B * NT, next);
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (v0 + b * NT < nvec) use(now[b], v0 + b * NT);
#pragma unroll
      for (int b = 0; b < B; ++b) now[b] = next[b];
    }
  };

  // pass 1: maximum and sum of 2^(c (x - max)) (0 for max while nothing is above -inf).
  // The difference comes first: fma(x, c, -(c max rounded)), one instruction less, has
  // the rounding of c max in it, which is any size where the maximum so far is a mask's
  // large number (and NaN follows from infinity times 0).
  const float c = (float)(1.4426950408889634 * it);
  float mx = -kInf, shift = 0.0f, sum = 0.0f;
  auto power = [&](float x, float of) { return __builtin_amdgcn_exp2f((x - of) * c); };
  auto taken = [&](int j) { return (bits[(j + skip) >> 5] >> ((j + skip) & 31)) & 1u; };
  auto more = [&](float hi) {
    if (hi > mx) {
      sum *= mx > -kInf ? power(mx, hi) : 1.0f;  // (a sum of nothing yet: 0, or NaN, which stays)
      mx = shift = hi;
    }
  };
  auto one = [&](int j) {
    if (rest && taken(j)) return;
    const float x = Z::value(z[j]);
    more(x);
    sum += power(x, shift);
  };
  for (int j = tid; j < head; j += NT) one(j);
  for (int j = tail0 + tid; j < V; j += NT) one(j);
  stream([&](const u4& v, int at) {
    float x[VE], hi = -kInf;
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = Vec<Z>::get(v, i);
    uint32_t out = 0;
    if (rest) out = bits[(vbase + at) * VE >> 5] >> ((vbase + at) * VE & 31) & ((1u << VE) - 1);
    if (out != 0) {
#pragma unroll
      for (int i = 0; i < VE; ++i) x[i] = (out >> i) & 1u ? -kInf : x[i];
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) hi = fmaxf(hi, x[i]);
    more(hi);
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < VE; ++i) part += power(x[i], shift);
    sum += part;
  });
  // a lane's, a wavefront's, then the workgroup's: sums in the unit of the larger
  // maximum (0 where nothing is above -inf). A NaN: fmax passes over it, the sum
  // does not.
  auto rescaled = [&](float s, float of, float to) {
    return of < to && s == s ? (of > -kInf ? s * power(of, to) : 0.0f) : s;
  };
  const float wtop = wave_max(mx);
  const float wtotal = wave_sum(rescaled(sum, mx, wtop));
  if (lane == 0) {
    wmax[w] = wtop;
    wsum[w] = wtotal;
  }
  __syncthreads();
  if (none_left) return zeros();
  const float top = wave_max(wmax[lane & (NW - 1)]);
  const float mine = rescaled(wsum[lane & (NW - 1)], wmax[lane & (NW - 1)], top);
  const double left = wave_sum(lane < NW ? (double)mine : 0.0);
  const float tshift = top > -kInf ? top : 0.0f;

  // the entries: the student's mass there, each index once (the lowest entry's), in
  // the unit of the largest logit of all, e^(ref / T); below: that of the sum, in it
  const double g = (double)weight * a.temperature * a.grad_scale;
  double total = left, ref = top, below = 0.0;
  if (w == own) {
    if (rest) {
      ref = fmaxf(top, wave_max(zmax));
      below = left > 0.0 ? ((double)top - ref) * it : 0.0;
    }
    double mass = 0.0;
#pragma unroll 1
    for (int i = lane; i < K; i += 64) {
      if (index[i] < 0) continue;
      const double v = exp(((double)zj[i] - ref) * it);
      e[i] = v;
      bool first = true;
      if (twice)
        for (int b = 0; b < i; ++b) first = first && index[b] != index[i];
      if (rest && first) mass += v;
    }
    if (rest) total = left * exp(below) + wave_sum(mass);
    // (left holds everything without a class for the rest; a student without mass
    // outside the entries has no gradient there, but a NaN's)
    const double Q = left * exp(below) / total;
    if (lane == 0) factor = (float)(rest ? (left == 0.0 ? 0.0 * total : g * (A * Q - P) / left) : g * A / total);
  }
  __syncthreads();
  if (w == own) {  // the loss, and the gradient at the entries, with the masses of all entries of an index
    double loss = 0.0;
    const double inverse = 1.0 / total;
#pragma unroll 1
    for (int i = lane; i < K; i += 64) {
      if (index[i] < 0) continue;
      const double pi = p[i] * pscale;
      if (pi != 0.0) loss += pi * (log(pi) - ((double)zj[i] - ref) * it);
      double all = pi;
      if (twice) {
        all = 0.0;
        for (int b = 0; b < K; ++b) all += index[b] == index[i] ? p[b] * pscale : 0.0;
      }
      e[i] = (A * e[i] * inverse - all) * g;
    }
    loss = wave_sum(loss);
    // the three logarithms side by side
    const double part = lane == 0 ? total : lane == 1 ? P : left, by = lane == 0 ? A : lane == 1 ? P : -P;
    const double whole = lane < 3 && by != 0.0 ? by * log(part) : 0.0;
    loss += wave_sum(whole);
    if (P != 0.0) loss -= P * below;
    if (lane == 0) {
      a.loss[m] = (float)(loss * ((double)weight * a.temperature * a.temperature));
    }
  }
  if (!dz) return;

  // pass 2
  const float cf = factor;
  auto grad = [&](float x) { return power(x, tshift) * cf; };
  for (int j = tid; j < head; j += NT) dz[j] = Z::pack(grad(Z::value(z[j])));
  for (int j = tail0 + tid; j < V; j += NT) dz[j] = Z::pack(grad(Z::value(z[j])));
  stream([&](const u4& v, int at) {
    float f[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = grad(Vec<Z>::get(v, i));
    __builtin_nontemporal_store(Vec<Z>::put(f), (u4*)(dz + head + at * VE));
  });
  __syncthreads();  // the entries' places have been written
  if (w == own) {
#pragma unroll 1
    for (int i = lane; i < K; i += 64)
      if (index[i] >= 0) dz[index[i]] = Z::pack((float)e[i]);
  }
}

}  // namespace

// Lanes per row. Many rows: as few as keep a CU's memory path busy with several
// rows, so that they cover each other's latencies; with a gradient the rows in flight
// have to stay in the memory-side cache until the second pass, so that long rows
// take more lanes (4096 bf16 rows with the rest and 256 / 512 / 1024 lanes: of 131072
// 623 / 510 / 482 us, of 32000 141 / 128 / 138, of 8000 39 / 49 / 71; the loss alone,
// of 131072 195 / 187 / 195, of 32000 65 / 66 / 88, of 8000 28 / 37 / 57). Few rows:
// the row itself is the latency (16 rows of 131072 44 / 30 / 24).
hipError_t launch_distill(const DistillArgs& a, int z_type, int value_type, hipStream_t stream) {
  with_type(z_type, [&](auto z) {
    typedef decltype(z) Z;
    constexpr int VE = Vec<Z>::VE;
    const unsigned lds = (unsigned)(a.K * 24 + (a.V + VE + 31) / 32 * 4);
    auto go = [&](auto kernel, int threads) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)a.M), dim3(threads), lds, stream, a, value_type);
    };
    const int kb = a.V / 1024 * (16 / VE);  // of a row
    const bool few = a.M <= 512;
    if (few ? kb >= 32 : a.dz && kb >= 192) go(distill_kernel<Z, 1024>, 1024);
    else if (few ? kb >= 8 : a.dz && kb >= 48) go(distill_kernel<Z, 512>, 512);
    else go(distill_kernel<Z, 256>, 256);
  });
  return hipGetLastError();
}

}  // namespace paro
