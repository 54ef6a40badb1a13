// gfx950 kernel for the experts' products where an expert has a few rows to some
// dozens: the weights are what has to be moved, and every expert's are read once
// (once per 16 TT rows).
//
// A workgroup owns up to 16 TT rows of one expert by 64 TC of its weight rows (gated:
// half of them gate rows, and the same channels' up rows), four wavefronts of 16 TC
// weight rows each, and goes over k in chunks of 128. Codes and X' come by
// load-to-LDS DMA into two stages, each an LDS object of its own; X' is shared by
// the wavefronts, so there is one barrier a chunk. Two to four workgroups fit a CU
// and keep its loads coming. (Three stages and fewer workgroups: the same bytes on
// their way, but longer rounds.)
// (w4_tiles_kernel, whose wavefronts share out k and meet in LDS, holds a CU alone
// and does nothing else while its operands arrive: 64 tokens, 8 of 64 experts,
// gated 2048 -> 1024, 80 us.)
//  * X' [16 TT rows][16 pieces of 8 channels], piece p of row t at p ^ t (low four
//    bits);
//  * codes of a wavefront [TC][16 rows][4 pieces of 32 codes], piece p of row r at
//    p ^ (r / 4): 16 lanes of an operand read touch every bank once.
// Scales and zeros: lane l has weight row l of its wavefront, four chunks' at a
// time in registers, and passes them on: a load touches a line per row, so that
// loads group by group keep the address path longer than the codes do (777 tokens,
// 4 of 60 experts, groups of 64, 1408 -> 2064: 74 us).
#include <algorithm>
#include <type_traits>

#include "expert_rows.h"
#include "paro_internal.h"
#include "w4_common.h"
#include "w4_epilogue.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

using namespace w4;

typedef __attribute__((address_space(3))) void lds_void;
constexpr int kRsrcWord3 = 0x00020000;  // gfx9 buffer resource word 3
constexpr int kWaitVmLgkm0 = 0x70;      // s_waitcnt vmcnt(0) lgkmcnt(0)
constexpr int kCus = 256;
// LDS bytes of a workgroup, and workgroups that fit a CU at once
constexpr int mid_lds(int tt, int tc) { return 2 * (4096 * tt + 4096 * tc); }
constexpr int mid_slots(int tt, int tc) { return 163840 / mid_lds(tt, tc) >= 4 ? 4 : 163840 / mid_lds(tt, tc); }

// GSH: log2(group / 64).
template <int EPI, int TT, int TC, int GSH, class ROWS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(mid_slots(TT, TC))))
void experts_mid_kernel(ROWS rows_of, const uint16_t* __restrict__ x, const uint8_t* __restrict__ qw,
                        const uint16_t* __restrict__ sc, const uint8_t* __restrict__ zr,
                        const uint16_t* __restrict__ bias, uint16_t* y, int N, int d, int nblk, const uint16_t* aux,
                        ActForm act, int erf) {
  constexpr bool GT = epi_gated(EPI);
  constexpr int CT = GT ? TC / 2 : TC;          // tiles of 16 output channels of a wavefront
  constexpr int XB = 4096 * TT, CB = 1024 * TC;  // bytes of a stage's X', and of a wavefront's codes
  __shared__ __attribute__((aligned(1024))) uint8_t X0[XB], X1[XB], C0[4 * CB], C1[4 * CB];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  ExpertTile tile;
  int nb;
  if (!rows_of.find_tile(blockIdx.x, 16 * TT, nblk, tile, nb)) return;
  const int m0 = tile.first, rows = tile.end - tile.first;
  const int P = GT ? 2 * N : N, half = d >> 1, groups = d >> (6 + GSH);
  const size_t first = (size_t)tile.expert * P;
  const int c0 = 16 * CT * (4 * nb + w);             // the wavefront's first output channel
  const bool any = c0 < N;  // (else it only fetches its share of X')
  const int left = any ? min(16 * CT, N - c0) : 1, base = any ? c0 : 0;
  const int segs = d >> 7;
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(x + (ROWS::kGather ? 0 : (size_t)m0 * d)), (short)0,
      (ROWS::kGather ? rows_tokens(rows_of) : rows) * d * 2, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rw =
      __builtin_amdgcn_make_buffer_rsrc((void*)(qw + first * half), (short)0, P * half, kRsrcWord3);
  // X' DMA t of wavefront w: rows 16 t + 4 w .. + 3 (past the end: the last one again)
  uint32_t xoff[4], woff[4];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int row = 16 * t + 4 * w + kq;
    xoff[t] = (uint32_t)(source_row(rows_of, m0, min(row, rows - 1)) * d * 2 + 16 * (r ^ (row & 15)));
  }
  // code DMA j: tile j's 16 rows
  auto weight_row = [&](int j, int row) { return base + min(16 * (j % CT) + row, left - 1) + (j / CT) * N; };
#pragma unroll
  for (int j = 0; j < TC; ++j) {
    const int row = lane >> 2;
    woff[j] = (uint32_t)(weight_row(j, row) * half + 16 * ((lane & 3) ^ (row >> 2)));
  }
  auto dma = [&](int c, uint8_t* xs, uint8_t* cs) {  // (past the last chunk: the last one again, never read)
    const int k = min(c, segs - 1);
    if (any) {
#pragma unroll
      for (int j = 0; j < TC; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(cs + CB * w + 1024 * j), 16, woff[j], 64 * k, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(xs + 4096 * t + 1024 * w), 16, xoff[t], 256 * k, 0, 0);
  };

  // scales and zeros of weight row `lane` of the wavefront, of four chunks: GQ
  // groups from any byte on, cut out of the aligned words that hold them (past the
  // last expert's weights: zero)
  constexpr int GQ = GSH == 0 ? 8 : GSH == 1 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc((void*)(sc + first * groups), (short)0, P * groups * 2, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rz =
      __builtin_amdgcn_make_buffer_rsrc((void*)(zr + first * groups), (short)0, P * groups, kRsrcWord3);
  const int srow = weight_row((lane >> 4) % TC, lane & 15) * groups;
  struct Scales {
    uint32_t s[5], z[3];  // the words
    uint32_t at;          // bytes to skip in them: zeros, scales << 8
  };
  auto load_scales = [&](int c, Scales& q) {  // c a multiple of 4
    const int g = srow + ((128 * c) >> (6 + GSH)), sa = (2 * g) & ~3, za = g & ~3;
    if constexpr (GQ == 2) {
      const uint2 sv = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rs, sa, 0, 0));
      const uint2 zv = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rz, za, 0, 0));
      q.s[0] = sv.x;
      q.s[1] = sv.y;
      q.z[0] = zv.x;
      q.z[1] = zv.y;
    } else {
      const u4 sv = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rs, sa, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) q.s[i] = sv[i];
      if constexpr (GQ == 8) {
        q.s[4] = __builtin_amdgcn_raw_buffer_load_b32(rs, sa + 16, 0, 0);
        const u4 zv = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rz, za, 0, 0));
#pragma unroll
        for (int i = 0; i < 3; ++i) q.z[i] = zv[i];
      } else {
        const uint2 zv = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rz, za, 0, 0));
        q.z[0] = zv.x;
        q.z[1] = zv.y;
      }
    }
    q.at = (uint32_t)(g & 3) | (uint32_t)((2 * g) & 3) << 8;
  };
  // the words cut so that the first scale and the first zero come first
  auto cut = [&](Scales& q) {
#pragma unroll
    for (int i = 0; i < GQ / 2; ++i) q.s[i] = __builtin_amdgcn_alignbyte(q.s[i + 1], q.s[i], q.at >> 8);
#pragma unroll
    for (int i = 0; i < (GQ + 3) / 4; ++i) q.z[i] = __builtin_amdgcn_alignbyte(q.z[i + 1], q.z[i], q.at & 3);
  };
  // group i of them: scale | zero << 16
  auto group_of = [&](const Scales& q, int i) {
    return ((q.s[i >> 1] >> (16 * (i & 1))) & 0xffffu) | ((q.z[i >> 2] >> (8 * (i & 3))) & 0xffu) << 16;
  };

  const uint32_t one = fp16_1024_pair();
  f4 acc[4][4];
#pragma unroll
  for (int j = 0; j < TC; ++j)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[j][t] = f4{0.f, 0.f, 0.f, 0.f};
  const int used = (rows + 15) >> 4;  // blocks of 16 rows that there are

  // chunk c, the cq-th of its four
  auto compute = [&](const uint8_t* xs, const uint8_t* cs, const Scales& q, int cq) {
    uint32_t mine, second = 0;
    if constexpr (GSH == 0) {
      mine = cq == 0 ? group_of(q, 0) : cq == 1 ? group_of(q, 2) : cq == 2 ? group_of(q, 4) : group_of(q, 6);
      second = cq == 0 ? group_of(q, 1) : cq == 1 ? group_of(q, 3) : cq == 2 ? group_of(q, 5) : group_of(q, 7);
    } else if constexpr (GSH == 1) {
      mine = cq == 0 ? group_of(q, 0) : cq == 1 ? group_of(q, 1) : cq == 2 ? group_of(q, 2) : group_of(q, 3);
    } else {
      mine = cq < 2 ? group_of(q, 0) : group_of(q, 1);
    }
    u4 v[4];
    h2 ss[4], zz[4], zz64[4];
#pragma unroll
    for (int j = 0; j < TC; ++j) {
      uint32_t sz = __shfl((int)mine, 16 * j + r);
      if constexpr (GSH == 0) {
        const uint32_t other = __shfl((int)second, 16 * j + r);
        sz = kq >= 2 ? other : sz;
      }
      v[j] = *(const u4*)(cs + CB * w + 1024 * j + 64 * r + 16 * (kq ^ (r >> 2)));
      ss[j] = splat2(__builtin_bit_cast(_Float16, (uint16_t)(sz & 0xffffu)));
      const float zf = (float)(sz >> 16);
      zz[j] = splat2((_Float16)(1024.0f + zf));
      zz64[j] = splat2((_Float16)(64.0f + zf));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h8 b[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < used) b[t] = *(const h8*)(xs + 4096 * t + 256 * r + 16 * ((4 * kq + i) ^ r));
#pragma unroll
      for (int j = 0; j < TC; ++j) {
        const h8 a = dequant8(v[j][i], zz[j], zz64[j], ss[j], one);
#pragma unroll
        for (int t = 0; t < TT; ++t)
          if (t < used) acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[t], acc[j][t], 0, 0, 0);
      }
    }
  };
  Scales now, next;
  if (any) load_scales(0, now);
  dma(0, X0, C0);
  // chunk c in (xs, cs); the other stage, which nobody reads after the barrier,
  // takes chunk c + 1
  auto chunk = [&](int c, uint8_t* xs, uint8_t* cs, uint8_t* xn, uint8_t* cn) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    dma(c + 1, xn, cn);
    if (!any) return;
    if ((c & 3) == 0) {
      if (c) now = next;
      cut(now);
      if (c + 4 < segs) load_scales(c + 4, next);
    }
    compute(xs, cs, now, c & 3);
  };
  int c = 0;
  for (; c + 2 <= segs; c += 2) {
    chunk(c, X0, C0, X1, C1);
    chunk(c + 1, X1, C1, X0, C0);
  }
  if (c < segs) chunk(c, X0, C0, X1, C1);
  __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);  // (the last DMA lands before the workgroup's LDS is another's)

  // acc[j][t][e] = Z[row m0 + 16 t + r][weight row 16 j + 4 kq + e of the wavefront]
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int m = m0 + 16 * t + r;
    if (m < tile.end) {
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        const int n = c0 + 16 * j + 4 * kq;
        if (n < N) {
          const uint16_t* b = bias ? bias + first : nullptr;
          if constexpr (EPI == kEpiShare) {
            epi_share(acc[j][t], rows_of.weight(m), m, n, N, b, (float*)y);
          } else {
            f4 z[2] = {acc[j][t], acc[GT ? j + CT : j][t]};
            epi_lane<EPI>(z, m, n, N, b, aux, act, erf, y);
          }
        }
      }
    }
  }
}

template <int EPI, int TT, int TC, int GSH>
hipError_t launch(const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                  const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N, int64_t d, const W4Epilogue& ep,
                  hipStream_t stream) {
  typedef ExpertRows<EPI != kEpiShare> Rows;
  const int64_t P = epi_gated(EPI) ? 2 * N : N, nblk = (P + 64 * TC - 1) / (64 * TC);
  const int64_t tiles = nblk * expert_blocks(t, 16 * TT);
  hipLaunchKernelGGL((experts_mid_kernel<EPI, TT, TC, GSH, Rows>), dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(256), 0,
                     stream, Rows{t}, x, qweight, scales, zeros, bias, (uint16_t*)y, (int)N, (int)d, (int)nblk, ep.aux,
                     act_form(ep.act), (int)(ep.act == PARO_ACT_GELU));
  return hipGetLastError();
}

template <int EPI, int TT, int TC>
hipError_t launch_group(const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                        const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N, int64_t d, int group,
                        const W4Epilogue& ep, hipStream_t stream) {
  auto go = group == 64 ? launch<EPI, TT, TC, 0> : group == 128 ? launch<EPI, TT, TC, 1> : launch<EPI, TT, TC, 2>;
  return go(t, x, qweight, scales, zeros, bias, y, N, d, ep, stream);
}

// Rows per tile (blocks of 16) by the mean number of rows of an expert that has
// any; then the weight tiles of a wavefront: four, or two where that fills the
// rounds better.
struct Shape {
  int tt, tc;
  int64_t tiles;  // that are expected
};
Shape shape_of(const ExpertRouting& t, int64_t P) {
  const int64_t used = std::min<int64_t>(t.E, t.R);
  Shape s{t.R <= 8 * used ? 1 : t.R <= 20 * used ? 2 : 4, 4, 0};
  const int64_t blocks = std::max<int64_t>(used, t.R / (16 * s.tt) + used / 4);
  auto tiles = [&](int tc) { return blocks * ((P + 64 * tc - 1) / (64 * tc)); };
  auto rounds = [&](int tc) { return (tiles(tc) + kCus * mid_slots(s.tt, tc) - 1) / (kCus * mid_slots(s.tt, tc)); };
  if (rounds(2) * 6 <= rounds(4) * 10) s.tc = 2;
  s.tiles = tiles(s.tc);
  return s;
}

template <int EPI>
hipError_t launch_epi(const Shape& s, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                      const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N,
                      int64_t d, int group, const W4Epilogue& ep, hipStream_t stream) {
  auto go = s.tc == 4 ? (s.tt == 1 ? launch_group<EPI, 1, 4> : s.tt == 2 ? launch_group<EPI, 2, 4> : launch_group<EPI, 4, 4>)
                      : (s.tt == 1 ? launch_group<EPI, 1, 2> : s.tt == 2 ? launch_group<EPI, 2, 2> : launch_group<EPI, 4, 2>);
  return go(t, x, qweight, scales, zeros, bias, y, N, d, group, ep, stream);
}

}  // namespace

// Enough workgroups to share the CUs.
bool experts_mid_fit(const ExpertRouting& t, int64_t P) { return shape_of(t, P).tiles >= kCus / 2; }

hipError_t launch_w4_experts_mid(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                                 const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y,
                                 int64_t N, int64_t d, int group, const W4Epilogue& ep, hipStream_t stream) {
  auto go = epi == kEpiGated ? launch_epi<kEpiGated> : epi == kEpiGatedGrad ? launch_epi<kEpiGatedGrad>
                                                                            : launch_epi<kEpiShare>;
  return go(shape_of(t, epi_gated(epi) ? 2 * N : N), t, x, qweight, scales, zeros, bias, y, N, d, group, ep, stream);
}

}  // namespace paro
