// Shared pieces of the W4G128 kernels: vector types and the int4 -> fp16
// dequantization used by both the small-batch and the large-batch linear.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace paro {
namespace w4 {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// Packed codes: one 32-bit word per 8 consecutive channels c0 .. c7, the even
// channels in bits 0..15 and the odd ones in bits 16..31, 4 bits each in
// channel order (word = c0 | c2 << 4 | c4 << 8 | c6 << 12 | c1 << 16 | ...).
// Masking one nibble of each 16-bit half and OR-ing in the fp16 pattern of
// 1024.0 gives the pair (c_{2i}, c_{2i+1}) in channel order: with the mask
// 0x000F000F as v = 1024 + q, with 0x00F000F0 as v = 1024 + 16 q. Then v -
// (1024 + z) or, fused, v / 16 - (64 + z) is exactly q - z in packed fp16, and
// one packed multiply by s rounds (q - z) s once, to a subnormal too. (The
// sixteenth is taken of v and not of s: s / 16 is not exact below s = 2^-10.)
// Eight values cost one shift, four and-or and eight packed fp16 operations.
//
// zz = (1024 + z, 1024 + z), zz64 = (64 + z, 64 + z), ss = (s, s); `one` =
// 0x64006400 held in a vector register, so that each (w & mask) | one is a
// single v_and_or_b32 (the mask is then the only scalar operand, as gfx9
// encodings allow).
__device__ __forceinline__ h8 dequant8(uint32_t w, h2 zz, h2 zz64, h2 ss, uint32_t one) {
  const uint32_t w8 = w >> 8;
  const h2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  auto high = [&](uint32_t bits) {
    return __builtin_elementwise_fma(__builtin_bit_cast(h2, bits | one), sixteenth, -zz64) * ss;
  };
  const h2 v0 = (__builtin_bit_cast(h2, (w & 0x000F000Fu) | one) - zz) * ss;      // c0, c1
  const h2 v1 = high(w & 0x00F000F0u);                                            // c2, c3
  const h2 v2 = (__builtin_bit_cast(h2, (w8 & 0x000F000Fu) | one) - zz) * ss;     // c4, c5
  const h2 v3 = high(w8 & 0x00F000F0u);                                           // c6, c7
  h8 out;
  out[0] = v0.x;
  out[1] = v0.y;
  out[2] = v1.x;
  out[3] = v1.y;
  out[4] = v2.x;
  out[5] = v2.y;
  out[6] = v3.x;
  out[7] = v3.y;
  return out;
}

// The fp16 pattern pair of 1024.0 in a vector register (see dequant8).
__device__ __forceinline__ uint32_t fp16_1024_pair() {
  uint32_t v;
  asm volatile("v_mov_b32 %0, 0x64006400" : "=v"(v));
  return v;
}

__device__ __forceinline__ h2 splat2(_Float16 v) { return h2{v, v}; }
__device__ __forceinline__ float half_lo(uint32_t v) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(v & 0xffffu));
}
__device__ __forceinline__ float half_hi(uint32_t v) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(v >> 16));
}
__device__ __forceinline__ uint32_t half_bits(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
}

// Meeting of the `pieces` workgroups that share a tile's contraction, on one
// counter that is zero between calls: each stores its partial tile, then counts
// itself in here, and the last one to do so (true, in every thread) finds all
// of them stored and adds them. Nobody waits for another workgroup. sys: the
// workgroups may sit on different XCDs; slot: a word of LDS.
__device__ __forceinline__ bool arrive_last(uint32_t* cnt, int pieces, int sys, volatile uint32_t* slot) {
  __builtin_amdgcn_s_waitcnt(0);  // this wavefront's stores have reached L2 / memory
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t before = sys ? __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM)
                                : __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const bool last = before == (uint32_t)(pieces - 1);
    if (last) {  // (all have counted themselves in)
      if (sys) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
      else __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    *slot = last;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane((int)*slot) != 0;
}

}  // namespace w4
}  // namespace paro
