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

// Which kernel: the 256 x 256 tiles from a mean of 144 rows on (and for two k-tiles;
// below, most of a tile is empty), the rows' kernel, which works on a row's weights
// without the others', for few pairs in all, else the middle one. Microseconds of
// rows | middle and middle | wide:
//   gated 2048 -> 1024, 64 experts: 16 rows 12 | 13, 32 rows 18 | 17; a mean of 128
//     rows 112 | 124, 160 133 | 130, 256 201 | 191;
//   gated 4096 -> 4096, 16 experts: 4 rows 16 | 25, 8 rows 20 | 27, 16 rows 35 | 32;
//     96 176 | 183, 128 218 | 191, 256 402 | 314;
//   14336 <- 4096, 8 experts: 2 rows 22 | 27, 4 rows 32 | 30; 96 169 | 172, 128 210 |
//     191, 256 381 | 328;
//   1024 -> 512, 128 experts: 32 rows 13 | 12; 128 46 | 48, 256 74 | 84.
// (The rule for the tiles goes by rows alone: where an expert is as small as the last
// it is wrong still at 256 rows, by 13%, and where it is large it could begin at 128.)
hipError_t launch_w4_experts(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                             const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N,
                             int64_t d, int group, const W4Epilogue& ep, hipStream_t stream) {
  const int64_t P = epi_gated(epi) ? 2 * N : N;
  auto go = d >= 256 && t.R >= 144 * (int64_t)t.E          ? launch_w4_experts_wide
            : t.R * P <= 16 * d && t.R <= 4 * (int64_t)t.E ? launch_w4_experts_rows
                                                           : launch_w4_experts_mid;
  return go(epi, t, x, qweight, scales, zeros, bias, y, N, d, group, ep, stream);
}

}  // namespace paro
