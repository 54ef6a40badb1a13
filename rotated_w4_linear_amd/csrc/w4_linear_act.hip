// The large-batch W4 linear with bias, activation and residual (w4_epilogue.h).
#include "w4_gemm_kernels.h"

#pragma clang fp contract(off)

namespace paro {

hipError_t launch_w4_gemm_act(
    const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
    const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
    uint32_t* cnt, float* part, const W4Epilogue& ep, hipStream_t stream) {
  return launch_w4_gemm_epi<kEpiAct>(x, qweight, scales, zeros, bias, y, M, N, d, group, cnt, part, ep, stream);
}

}  // namespace paro
