// gfx950 kernel for the experts' products where an expert has from one row to some
// hundred: the weights are what has to be moved, and every expert's are read once
// (once per 16 TT rows).
//
// A workgroup owns up to 16 TT rows of one expert by 128 of its weight rows (gated:
// 64 gate rows, and the same channels' up rows), four wavefronts of 32 weight rows
// each, and goes over k in chunks of 128. Codes and X' come by load-to-LDS DMA into
// two stages, each an LDS object of its own; X' is shared by the wavefronts, so there
// is one barrier a chunk. Four workgroups fit a CU and keep its loads coming. Measured
// against it, gated 2048 -> 1024, 8 of 64 experts, 768 tokens (64 rows a tile, 90 us)
// and 16 (28 us): four stages, whose LDS leaves room for fewer workgroups, 161 and
// 29; 256 weight rows instead of 128, 99 and 38.
// (w4_tiles_kernel, whose wavefronts share out k and meet in LDS, holds a CU alone
// and does nothing else while its operands arrive: 64 tokens, 76 us for 32.)
// What bounds it: few rows, the stream of the weights (64 tokens: 133 MB in 33 us, 4.0
// TB/s); from a dozen rows of an expert on the waits for a chunk and the
// dequantization, each some 40% of the cycles (777 tokens below: 43 us).
//  * X' [16 TT rows][16 pieces of 8 channels], piece p of row t at p ^ t (low four
//    bits);
//  * codes of a wavefront [2 tiles][16 rows][4 pieces of 32 codes], piece p of row r at
//    p ^ (r / 4): 16 lanes of an operand read touch every bank once.
// Scales and zeros: lane l has weight row l of its wavefront, four chunks' at a
// time in registers, and passes them on: a load touches a line per row, so that
// loads group by group keep the address path longer than the codes do (777 tokens,
// 4 of 60 experts, groups of 64, 1408 -> 2064: 74 us, at the time, for 55).
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
constexpr int kSlots = 4;               // workgroups that fit a CU at once

// GSH: log2(group / 64).
template <int EPI, int TT, int GSH, class ROWS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(kSlots)))
void experts_mid_kernel(ROWS rows_of, const uint16_t* __restrict__ x, const uint8_t* __restrict__ qw,
                        const uint16_t* __restrict__ sc, const uint8_t* __restrict__ zr,
                        const uint16_t* __restrict__ bias, uint16_t* y, int N, int d, int nblk, const uint16_t* aux,
                        ActForm act, int erf) {
  constexpr bool GT = epi_gated(EPI);
  constexpr int TC = 2;                         // weight tiles of a wavefront
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
  // (past the last chunk: the last one again, never read)
  auto dma_x = [&](int c, uint8_t* xs, auto blocks) {
    const int k = min(c, segs - 1);
#pragma unroll
    for (int t = 0; t < decltype(blocks)::value; ++t)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(xs + 4096 * t + 1024 * w), 16, xoff[t], 256 * k, 0, 0);
  };
  auto dma = [&](int c, uint8_t* xs, uint8_t* cs, auto blocks) {
    const int k = min(c, segs - 1);
#pragma unroll
    for (int j = 0; j < TC; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(cs + CB * w + 1024 * j), 16, woff[j], 64 * k, 0, 0);
    dma_x(c, xs, blocks);
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

  // a chunk, the cq-th of its four, with so many blocks of 16 rows
  auto compute = [&](const uint8_t* xs, const uint8_t* cs, const Scales& q, int cq, auto blocks) {
    constexpr int U = decltype(blocks)::value;
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
      h8 b[4];
#pragma unroll
      for (int t = 0; t < U; ++t) b[t] = *(const h8*)(xs + 4096 * t + 256 * r + 16 * ((4 * kq + i) ^ r));
#pragma unroll
      for (int j = 0; j < TC; ++j) {
        const h8 a = dequant8(v[j][i], zz[j], zz64[j], ss[j], one);
#pragma unroll
        for (int t = 0; t < U; ++t) acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[t], acc[j][t], 0, 0, 0);
      }
    }
  };
  // the stage's chunk is there, and nobody reads the other stage any more
  auto sync = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // all chunks, with so many blocks of 16 rows (a loop for each: branches between the
  // products would cost more than they do)
  auto run = [&](auto blocks) {
    if (!any) {
      dma_x(0, X0, blocks);
      for (int c = 0; c < segs; ++c) {
        sync();
        dma_x(c + 1, c & 1 ? X0 : X1, blocks);
      }
      return;
    }
    Scales now, next;
    load_scales(0, now);
    dma(0, X0, C0, blocks);
    // chunk c + i in its stage, the other one takes chunk c + i + 1. (Four chunks,
    // which share their scales' loads, in a row and without a branch: the waits stay
    // where they are here.)
    auto chunk = [&](int c, auto at) {
      constexpr int i = decltype(at)::value;
      sync();
      dma(c + i + 1, i & 1 ? X0 : X1, i & 1 ? C0 : C1, blocks);
      if (i == 0) {
        cut(now);
        load_scales(min(c + 4, (segs - 1) & ~3), next);
      }
      compute(i & 1 ? X1 : X0, i & 1 ? C1 : C0, now, i, blocks);
    };
    int c = 0;
    for (; c + 4 <= segs; c += 4) {
      chunk(c, std::integral_constant<int, 0>{});
      chunk(c, std::integral_constant<int, 1>{});
      chunk(c, std::integral_constant<int, 2>{});
      chunk(c, std::integral_constant<int, 3>{});
      now = next;
    }
    if (c < segs) chunk(c, std::integral_constant<int, 0>{});
    if (c + 1 < segs) chunk(c, std::integral_constant<int, 1>{});
    if (c + 2 < segs) chunk(c, std::integral_constant<int, 2>{});
  };
  if (TT > 1 && rows > 32) run(std::integral_constant<int, TT>{});
  else if (TT > 1 && rows > 16) run(std::integral_constant<int, TT < 2 ? TT : 2>{});
  else run(std::integral_constant<int, 1>{});
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

template <int EPI, int TT, int GSH>
hipError_t launch(const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                  const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N, int64_t d, const W4Epilogue& ep,
                  hipStream_t stream) {
  typedef ExpertRows<EPI != kEpiShare> Rows;
  const int64_t P = epi_gated(EPI) ? 2 * N : N, nblk = (P + 127) / 128;
  const int64_t tiles = nblk * expert_blocks(t, 16 * TT);
  hipLaunchKernelGGL((experts_mid_kernel<EPI, TT, GSH, Rows>), dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(256), 0,
                     stream, Rows{t}, x, qweight, scales, zeros, bias, (uint16_t*)y, (int)N, (int)d, (int)nblk, ep.aux,
                     act_form(ep.act), (int)(ep.act == PARO_ACT_GELU));
  return hipGetLastError();
}

template <int EPI, int TT>
hipError_t launch_group(const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                        const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N, int64_t d, int group,
                        const W4Epilogue& ep, hipStream_t stream) {
  auto go = group == 64 ? launch<EPI, TT, 0> : group == 128 ? launch<EPI, TT, 1> : launch<EPI, TT, 2>;
  return go(t, x, qweight, scales, zeros, bias, y, N, d, ep, stream);
}

// Rows per tile (blocks of 16) by the mean number of an expert's rows: a tile's rows
// share the dequantization, which is most of the work from a dozen rows on. 16 | 32 |
// 48 | 64 rows, microseconds, random numbers of rows:
//   gated 2048 -> 1024, 64 experts: a mean of 12 32 | 31 | 34 | 39, 24 45 | 44 | 44 |
//     51, 48 - | 62 | 59 | 61, 96 - | 97 | 90 | 90;
//   gated 4096 -> 14336, 8 experts: 12 148 | 118 | 122 | 132, 32 - | 179 | 171 | 188,
//     64 - | 274 | 235 | 234;
//   1024 -> 512, 128 experts: 12 20 | 21 | 21 | 23, 32 - | 25 | 25 | 28, 96 - | 39 | 39 | 43.
template <int EPI>
hipError_t launch_epi(const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                      const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N, int64_t d, int group,
                      const W4Epilogue& ep, hipStream_t stream) {
  const int64_t E = t.E;
  auto go = t.R <= 8 * E ? launch_group<EPI, 1> : t.R <= 32 * E ? launch_group<EPI, 2> : launch_group<EPI, 3>;
  return go(t, x, qweight, scales, zeros, bias, y, N, d, group, ep, stream);
}

}  // namespace

hipError_t launch_w4_experts_mid(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                                 const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y,
                                 int64_t N, int64_t d, int group, const W4Epilogue& ep, hipStream_t stream) {
  auto go = epi == kEpiGated ? launch_epi<kEpiGated> : epi == kEpiGatedGrad ? launch_epi<kEpiGatedGrad>
                                                                            : launch_epi<kEpiShare>;
  return go(t, x, qweight, scales, zeros, bias, y, N, d, group, ep, stream);
}

}  // namespace paro
