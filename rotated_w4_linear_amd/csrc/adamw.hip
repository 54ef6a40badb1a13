// gfx950 kernel for one AdamW step over many tensors at once:
//   m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2,
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32, every operation rounded on its own. A pass over memory: with fp32
// parameters and gradients 28 bytes per value, 16.06 with 8-bit moments.
//
// 8-bit moments: m and r = sqrt(v) (the form the update uses; v itself spans
// twice the exponent range) as e4m3 numbers times one fp32 scale per block of
// 256 consecutive values of a tensor, scale = largest magnitude / 448. The
// scale is not a power of two: the largest value of a block is then kept to
// fp32 accuracy, so that slow decays, which are far below half a step of
// e4m3, still act, through the scale. r is never rounded to zero where v is
// not: a lost r would turn m / (r + eps) into a jump.
//
// One workgroup takes a chunk of 2048 values of one tensor, each wavefront two
// blocks of 256, each lane four consecutive values of a block (16-byte
// accesses of fp32). Up to kAdamTensors tensors' pointers travel as kernel
// arguments; longer lists lie in a table that is uploaded once, so that a step
// is one launch (448 angle and scale tensors of 32 layers, 6.1 M values: 44.5
// us in four launches, 31.6 in one, 5.4 TB/s) and needs no upload.
#include <cstring>

#include "paro_internal.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: a block below it is held as zero

template <int TYPE>  // PARO_TYPE_*
__device__ __forceinline__ float to_f32(uint32_t bits) {
  if constexpr (TYPE == PARO_TYPE_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  else return __builtin_bit_cast(float, bits << 16);
}
template <int TYPE>
__device__ __forceinline__ uint32_t from_f32(float f) {
  if constexpr (TYPE == PARO_TYPE_F16) return __builtin_bit_cast(uint16_t, (_Float16)f);
  else return __builtin_bit_cast(uint16_t, (__bf16)f);
}

// values i .. i + 3 of a tensor of n (zeros past its end)
template <int TYPE>
__device__ __forceinline__ f4 load4(const void* base, int64_t i, int64_t n, bool vec) {
  f4 o = {0.f, 0.f, 0.f, 0.f};
  if constexpr (TYPE == PARO_TYPE_F32) {
    const float* p = (const float*)base + i;
    if (vec && i + 4 <= n) return *(const f4*)p;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) o[e] = p[e];
  } else {
    const uint16_t* p = (const uint16_t*)base + i;
    if (vec && i + 4 <= n) {
      const u2 r = *(const u2*)p;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = to_f32<TYPE>((r[e >> 1] >> (16 * (e & 1))) & 0xffffu);
      return o;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) o[e] = to_f32<TYPE>(p[e]);
  }
  return o;
}
template <int TYPE>
__device__ __forceinline__ void store4(void* base, int64_t i, int64_t n, bool vec, f4 v) {
  if constexpr (TYPE == PARO_TYPE_F32) {
    float* p = (float*)base + i;
    if (vec && i + 4 <= n) {
      *(f4*)p = v;
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) p[e] = v[e];
  } else {
    uint16_t* p = (uint16_t*)base + i;
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = from_f32<TYPE>(v[e]);
    if (vec && i + 4 <= n) {
      *(u2*)p = u2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) p[e] = (uint16_t)h[e];
  }
}

// four e4m3 values in a word
__device__ __forceinline__ f4 from_e4m3(uint32_t w) {
  return f4{__builtin_amdgcn_cvt_f32_fp8(w, 0), __builtin_amdgcn_cvt_f32_fp8(w, 1),
            __builtin_amdgcn_cvt_f32_fp8(w, 2), __builtin_amdgcn_cvt_f32_fp8(w, 3)};
}
__device__ __forceinline__ uint32_t to_e4m3(f4 v) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
}

// largest magnitude over the wavefront's 64 x 4 values; compared as bit
// patterns, which order non-negative floats and put NaN above infinity, so
// that a NaN or infinity of a block shows in its scale
__device__ __forceinline__ float block_max(f4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f = v[e];
    m = max(m, __builtin_bit_cast(uint32_t, f) & 0x7fffffffu);
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s));
  return __builtin_bit_cast(float, m);
}

// the tensor of a chunk: the last one that starts at or before it
__device__ __forceinline__ AdamwTensor find(const AdamwLaunch& a, uint32_t chunk, int lane) {
  int ti = -1;
#pragma unroll
  for (int h = 0; h < (kAdamTensors + 63) / 64; ++h) {
    const int i = 64 * h + lane;
    const bool le = i < a.count && a.t[i < kAdamTensors ? i : 0].chunk0 <= chunk;
    ti += __popcll(__ballot(le));
  }
  return a.t[__builtin_amdgcn_readfirstlane(ti)];
}
__device__ __forceinline__ AdamwTensor find(const AdamwTable& a, uint32_t chunk, int) { return a.t[a.of_chunk[chunk]]; }

template <int PT, int GT, bool EIGHT, class Args>
__global__ __launch_bounds__(256) void adamw_kernel(Args args) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const AdamwScalars& a = args.s;
  const uint32_t chunk = blockIdx.x;
  const AdamwTensor t = find(args, chunk, lane);
  const int64_t base = (int64_t)(chunk - t.chunk0) * kAdamChunk + w * 512;
  if (base >= t.n) return;
  const bool pv = ((uintptr_t)t.p & (PT == PARO_TYPE_F32 ? 15 : 7)) == 0;
  const bool gv = ((uintptr_t)t.g & (GT == PARO_TYPE_F32 ? 15 : 7)) == 0;
  const int64_t state0 = (int64_t)t.block0 * 256;

  f4 p[2], g[2], m[2], v[2];
  uint32_t mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
  float ms[2] = {0.f, 0.f}, vs[2] = {0.f, 0.f};
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t i = base + 256 * b + 4 * lane;
    if (base + 256 * b >= t.n) continue;
    // (the moments are padded to whole blocks: their loads need no bound)
    if constexpr (EIGHT) {
      mc[b] = *(const uint32_t*)((const uint8_t*)a.m + state0 + i);
      vc[b] = *(const uint32_t*)((const uint8_t*)a.v + state0 + i);
      const int64_t blk = (int64_t)t.block0 + (base >> 8) + b;
      ms[b] = a.ms[blk];
      vs[b] = a.vs[blk];
    } else {
      m[b] = *(const f4*)((const float*)a.m + state0 + i);
      v[b] = *(const f4*)((const float*)a.v + state0 + i);
    }
    g[b] = load4<GT>(t.g, i, t.n, gv);
    p[b] = load4<PT>(t.p, i, t.n, pv);
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t i = base + 256 * b + 4 * lane;
    if (base + 256 * b >= t.n) break;  // (uniform: whole blocks)
    if constexpr (EIGHT) {
      m[b] = from_e4m3(mc[b]) * ms[b];
      const f4 r = from_e4m3(vc[b]) * vs[b];
      v[b] = r * r;
    }
    f4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[b][e] = m[b][e] * a.b1 + g[b][e] * a.c1;
      v[b][e] = v[b][e] * a.b2 + g[b][e] * g[b][e] * a.c2;
      r[e] = __builtin_sqrtf(v[b][e]);
      p[b][e] = p[b][e] * a.keep - (m[b][e] / (r[e] * a.root + a.eps)) * a.rate;
    }
    store4<PT>((void*)t.p, i, t.n, pv, p[b]);
    if constexpr (EIGHT) {
      // (values past the tensor's end are zero and stay so)
      float tm = block_max(m[b]), tr = block_max(r);
      if (tm < kTiny) tm = 0.0f;
      if (tr < kTiny) tr = 0.0f;
      const float im = tm == 0.0f ? 0.0f : (1.0f / tm) * kE4m3Max;
      const float ir = tr == 0.0f ? 0.0f : (1.0f / tr) * kE4m3Max;
      const uint32_t cm = to_e4m3(m[b] * im);
      uint32_t cr = to_e4m3(r * ir);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v[b][e] > 0.0f && tr > 0.0f && ((cr >> (8 * e)) & 0xffu) == 0) cr |= 1u << (8 * e);
      *(uint32_t*)((uint8_t*)a.m + state0 + i) = cm;
      *(uint32_t*)((uint8_t*)a.v + state0 + i) = cr;
      if (lane == 0) {
        const int64_t blk = (int64_t)t.block0 + (base >> 8) + b;
        a.ms[blk] = tm * (1.0f / kE4m3Max);
        a.vs[blk] = tr * (1.0f / kE4m3Max);
      }
    } else {
      store4<PARO_TYPE_F32>((float*)a.m + state0, i, t.n, true, m[b]);
      store4<PARO_TYPE_F32>((float*)a.v + state0, i, t.n, true, v[b]);
    }
  }
}

template <int PT, int GT, class Args>
hipError_t launch_types(const Args& a, uint32_t chunks, bool eight, hipStream_t stream) {
  static_assert(sizeof(Args) <= 4096, "kernel arguments");
  if (eight) hipLaunchKernelGGL((adamw_kernel<PT, GT, true, Args>), dim3(chunks), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((adamw_kernel<PT, GT, false, Args>), dim3(chunks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <int PT, class Args>
hipError_t launch_param(const Args& a, uint32_t chunks, int gt, bool eight, hipStream_t stream) {
  switch (gt) {
    case PARO_TYPE_F32: return launch_types<PT, PARO_TYPE_F32>(a, chunks, eight, stream);
    case PARO_TYPE_F16: return launch_types<PT, PARO_TYPE_F16>(a, chunks, eight, stream);
    default: return launch_types<PT, PARO_TYPE_BF16>(a, chunks, eight, stream);
  }
}

template <class Args>
hipError_t launch_any(const Args& a, uint32_t chunks, int pt, int gt, bool eight, hipStream_t stream) {
  if (chunks == 0) return hipSuccess;
  switch (pt) {
    case PARO_TYPE_F32: return launch_param<PARO_TYPE_F32>(a, chunks, gt, eight, stream);
    case PARO_TYPE_F16: return launch_param<PARO_TYPE_F16>(a, chunks, gt, eight, stream);
    default: return launch_param<PARO_TYPE_BF16>(a, chunks, gt, eight, stream);
  }
}

}  // namespace

hipError_t launch_adamw(const AdamwLaunch& a, uint32_t chunks, int param_type, int grad_type, bool eight,
                        hipStream_t stream) {
  return launch_any(a, chunks, param_type, grad_type, eight, stream);
}
hipError_t launch_adamw(const AdamwTable& a, uint32_t chunks, int param_type, int grad_type, bool eight,
                        hipStream_t stream) {
  return launch_any(a, chunks, param_type, grad_type, eight, stream);
}

}  // namespace paro
