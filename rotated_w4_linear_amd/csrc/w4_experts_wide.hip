// The experts' products in 256 x 256 tiles (w4_gemm_kernels.h).
#include "w4_gemm_kernels.h"

#pragma clang fp contract(off)

namespace paro {

hipError_t launch_w4_experts_wide(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                                  const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y,
                                  int64_t N, int64_t d, int group, const W4Epilogue& ep, hipStream_t stream) {
  auto go = epi == kEpiGated       ? launch_w4_experts_wide_epi<kEpiGated, true>
            : epi == kEpiGatedGrad ? launch_w4_experts_wide_epi<kEpiGatedGrad, true>
                                   : launch_w4_experts_wide_epi<kEpiShare, false>;
  return go(t, x, qweight, scales, zeros, bias, y, N, d, group, ep, stream);
}

// Whether the products are taken in these tiles: two k-tiles at a time, and
// experts of enough rows.
bool experts_wide_fit(const ExpertRouting& t, int64_t P, int64_t d) {
  return d >= 256 && t.R >= 64 * (int64_t)t.E;
}

hipError_t launch_w4_experts(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                             const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N,
                             int64_t d, int group, const W4Epilogue& ep, hipStream_t stream) {
  const int64_t P = epi_gated(epi) ? 2 * N : N;
  auto go = experts_wide_fit(t, P, d)   ? launch_w4_experts_wide
            : experts_rows_fit(t) == 1  ? launch_w4_experts_rows
            : experts_mid_fit(t, P)     ? launch_w4_experts_mid
            : experts_rows_fit(t)       ? launch_w4_experts_rows
                                                                : launch_w4_experts_tiles;
  return go(epi, t, x, qweight, scales, zeros, bias, y, N, d, group, ep, stream);
}

}  // namespace paro
