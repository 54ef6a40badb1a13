// The small-batch gated W4 product act(Zg + bg) (Zu + bu) (w4_epilogue.h).
#include "w4_decode_kernels.h"

#pragma clang fp contract(off)

namespace paro {

hipError_t launch_w4_decode_gated(
    const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
    const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
    const paro_rotation* r, void* ws, const W4Epilogue& ep, hipStream_t stream) {
  return launch_w4_decode_epi<kEpiGated>(x, qweight, scales, zeros, bias, y, M, N, d, group, r, ws, ep, stream);
}

}  // namespace paro
