// The large-batch W4 linear without an epilogue of its own (w4_gemm_kernels.h),
// and the choice of kernel and split that every epilogue shares.
#include "w4_gemm_kernels.h"

#pragma clang fp contract(off)

namespace paro {

SmallGemm small_gemm(int64_t M, int64_t N, int64_t d) {
  SmallGemm g;
  g.nblk256 = (int)((N + GB_N - 1) / GB_N);
  g.half = (int64_t)g.nblk256 * ((M + 127) / 128) < kHalfTileBelow;
  const int gbm = g.half ? 64 : 128;
  g.mblk = (int)((M + gbm - 1) / gbm);
  g.narrow = g.half && (int64_t)g.nblk256 * g.mblk < kNarrowTileBelow;
  g.nblk = g.narrow ? (int)((N + GB_N / 2 - 1) / (GB_N / 2)) : g.nblk256;
  g.tiles = (int64_t)g.nblk * g.mblk;
  const int64_t kt = d / GB_K;
  const bool ks2 = g.tiles < 512 && kt % 2 == 0 && kt >= 4;
  const bool ks4 = g.narrow && kt % 4 == 0 && kt >= 16;
  g.ksin = ks4 ? 4 : ks2 ? 2 : 1;
  // with 64 x 128 tiles (and k split four ways inside) that leave CUs idle:
  // up to 4 workgroups per tile, each group of wavefronts keeping at least
  // kMinNarrowSplitKT k-tiles
  g.nsplit = 1;
  if (g.narrow && g.ksin == 4)
    while (g.nsplit < 4 && g.tiles * 2 * g.nsplit <= 256 && kt % (g.ksin * 2 * g.nsplit) == 0 &&
           kt / (g.ksin * 2 * g.nsplit) >= kMinNarrowSplitKT && g.tiles <= (int64_t)(kDecodeCounterBytes / 4))
      g.nsplit *= 2;
  return g;
}


GemmPlan plan_w4_gemm(int64_t M, int64_t N, int64_t d) {
  GemmPlan p;
  const int64_t nblk = (N + GB_N - 1) / GB_N, mblkw = (M + GW_M - 1) / GW_M;
  const int64_t tiles = nblk * mblkw, kt = d / GB_K;
  if (M <= kDecodeMaxM || d > (int64_t(1) << 21) || kt % 2 || d < 4 * GB_K) return p;
  // one tile per workgroup from kWideMinTiles tiles (stream-K measured slower
  // there: 2048 x 4096 -> 14336, 448 tiles, 252 against 223 us, the
  // workgroups of an XCD no longer reading the same k-tiles at the same
  // time); below, stream-K when every XCD holds n-blocks
  if (tiles >= kWideMinTiles) {
    p.wide = true;
    return p;
  }
  const int64_t nbmin = nblk / 8, nbmax = (nblk + 7) / 8;
  // Workgroups per XCD: the fewest k-tiles per range on the busiest XCD,
  // counting kSkMisaligned more for ranges that do not cut the tiles into
  // equal pieces (nor hold whole tiles): their pieces start at different k,
  // so the workgroups of an XCD stop sharing k-tiles in L2 (measured: 1300 x
  // 8192 -> 4096, 96 tiles of 128 k-tiles, 123 us with ranges of 48 against
  // 113 with 24 workgroups per XCD taking half tiles). Every range keeps at
  // least two k-tiles on the least busy XCD and kMinSplitKT on the busiest;
  // ranges of whole tiles (one tile per workgroup on fewer workgroups than
  // CUs) are not taken, nor misaligned ones on fewer than 3/4 of the CUs.
  int best = 0;
  int64_t best_cost = 0;
  for (int sl = kSkSlots; nbmin >= 1 && sl >= kSkSlots / 2; sl -= 4) {
    const int64_t units = nbmax * mblkw * kt;
    if (nbmin * mblkw * kt < 2 * sl) continue;
    const int64_t U = (units + sl - 1) / sl;
    if (U < kMinSplitKT || U % kt == 0) continue;  // (whole tiles: fewer workgroups than CUs)
    const bool aligned = units % (2 * sl) == 0 && kt % U == 0;
    if (!aligned && sl < kSkSlots * 3 / 4) continue;
    const int64_t cost = U + (aligned ? 0 : kSkMisaligned);
    if (!best || cost < best_cost) {
      best = sl;
      best_cost = cost;
    }
  }
  if (best) {
    p.wide = p.sk = true;
    p.sk_slots = best;
    p.partial_bytes = (size_t)8 * kSkSlots * 2 * GW_M * GB_N * 4;
    return p;
  }
  const SmallGemm g = small_gemm(M, N, d);
  if (g.nsplit > 1) {
    p.nsplit = g.nsplit;
    p.partial_bytes = (size_t)g.tiles * g.nsplit * 64 * 128 * 4;
  }
  return p;
}

void sk_shape(int64_t nblk, int64_t mblkw, int64_t L, int gsh, int slots, int64_t* panel_groups, bool* one_tile) {
  auto span = [&](int64_t kt0, int64_t KT) { return ((kt0 + KT - 1) >> gsh) - ((kt0 >> gsh) & ~int64_t(7)) + 1; };
  int64_t most = 0;
  bool one = true;
  for (int64_t x = 0; x < 8; ++x) {
    const int64_t nbx = (nblk - x + 7) / 8;
    if (nbx <= 0) continue;
    const int64_t H = nbx * mblkw * L / 2;
    for (int64_t j = 0; j < slots; ++j) {
      const int64_t s = 2 * (j * H / slots), e = 2 * ((j + 1) * H / slots);
      if (e <= s) continue;
      const int64_t t = s / L, k0 = s - t * L, te = (e - 1) / L;
      one = one && te == t;
      most = std::max(most, span(k0, std::min(L - k0, e - s)));
      if (te > t) most = std::max(most, span(0, e - te * L));
      if (te > t + 1 || (te > t && k0 == 0)) most = std::max(most, span(0, L));
    }
  }
  *panel_groups = most;
  *one_tile = one;
}

hipError_t launch_w4_gemm(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                          const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M,
                          int64_t N, int64_t d, int group, uint32_t* cnt, float* part, hipStream_t stream) {
  return launch_w4_gemm_epi<kEpiPlain>(x, qweight, scales, zeros, bias, y, M, N, d, group, cnt, part, W4Epilogue{},
                                       stream);
}

}  // namespace paro
