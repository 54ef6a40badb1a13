// The element types of a paro_type as the kernels load and store them.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/paro.h"

namespace paro {

struct F32 {
  typedef float raw;
  static __device__ __forceinline__ float value(raw v) { return v; }
  static __device__ __forceinline__ raw pack(float v) { return v; }
};
struct F16 {
  typedef uint16_t raw;
  static __device__ __forceinline__ float value(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ raw pack(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct BF16 {
  typedef uint16_t raw;
  static __device__ __forceinline__ float value(raw v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
  static __device__ __forceinline__ raw pack(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};

// go(F32{}), go(F16{}) or go(BF16{})
template <class Go>
void with_type(int type, Go go) {
  if (type == PARO_TYPE_F32) go(F32{});
  else if (type == PARO_TYPE_F16) go(F16{});
  else go(BF16{});
}

}  // namespace paro
