// gfx950 kernel for the W4 products with an epilogue (w4_epilogue.h) on a few
// tokens to a few hundred, where tiles of 64 x 128 and more leave CUs idle.
//
// A workgroup owns a small tile, 16 TT tokens by 16 TC weight rows, over the
// whole of k, which its wavefronts share out in chunks of 128; the sums meet in
// LDS, with no partial sums in memory and no counters. (Against the kernels that
// split k over workgroups: 14336 -> 4096 at 64 tokens 54 against 25 us, at 128
// tokens 48 against 36; gated 4096 -> 14336 at 64 tokens 58 against 36.) A CU's
// time is that of its operands' way through L2 and LDS: 64 x 64 tiles move 20 KB
// per chunk in 0.36 - 0.47 us, in which the matrix cores are busy for 0.11 us
// and the dequantization's vector instructions for 0.09 us.
//
// Operands go from global memory straight into LDS (16-byte load-to-LDS DMA),
// into a region of the wavefront's own, so no barrier is needed before they are
// read, and the loads of all wavefronts are in flight at once (half as many
// wavefronts with two chunks each, the next one's loads sent before the
// products: 4096 -> 4096 at 64 tokens 10.2 against 10.1 us, 64 x 64 tiles 22
// against 17.6, one wavefront per SIMD):
//  * X' [16 TT tokens][16 pieces of 8 channels], piece p of token t at p ^ t
//    (low four bits);
//  * codes [TC][16 rows][4 pieces of 32 codes], piece p of row r at
//    p ^ (r / 4): 16 lanes of an operand read touch every bank once.
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
constexpr int kWaitLgkm0 = 0xC07F;      // lgkmcnt(0) alone

// compute units: 32 in each of 8 XCDs
constexpr int kCus = 256;

// LDS bytes of a wavefront, and wavefronts per workgroup at most
constexpr int tile_bytes(int tt, int tc) { return 4096 * tt + 1024 * tc; }
constexpr int tile_waves(int tt, int tc) {
  return 163840 / tile_bytes(tt, tc) >= 16 ? 16 : 163840 / tile_bytes(tt, tc);
}

// EPI as in w4_epilogue.h. Gated: half of the TC weight tiles are the gate's,
// the others the same channels of the up projection.
template <int EPI, int TT, int TC>
__global__ __launch_bounds__(64 * tile_waves(TT, TC))
void w4_tiles_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ qw,
                     const uint16_t* __restrict__ sc, const uint8_t* __restrict__ zr,
                     const uint16_t* __restrict__ bias, uint16_t* y, int M, int N, int d, int gsh, int mblk,
                     int blocks, int per, const uint16_t* aux, ActForm act, int erf) {
  constexpr bool GT = epi_gated(EPI);
  constexpr int CT = GT ? TC / 2 : TC;  // tiles of 16 output channels
  constexpr int WB = tile_bytes(TT, TC);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[tile_waves(TT, TC) * WB];
  // the token blocks of a channel block on one XCD, one after the other: they
  // share its weights
  const int blk = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (blk >= blocks) return;
  const int nb = blk / mblk;
  const int m0 = 16 * TT * (blk - nb * mblk), c0 = 16 * CT * nb;
  const int lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), nw = blockDim.x >> 6;
  const int segs = d >> 7, sgr = d >> (6 + gsh);  // chunks; quantization groups per row
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc((void*)(x + (size_t)m0 * d), (short)0,
                                                                      min(16 * TT, M - m0) * d * 2, kRsrcWord3);
  const int rows = min(16 * CT, N - c0);  // rows past N repeat the last one and are never stored
  auto codes = [&](int up) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)(qw + ((size_t)up * N + c0) * (size_t)(d >> 1)), (short)0,
                                             rows * (d >> 1), kRsrcWord3);
  };
  uint32_t xoff[16], woff[4];  // (not sized by TT and TC: the host pass could not instantiate the loads)
#pragma unroll
  for (int t = 0; t < 4 * TT; ++t) {
    const int row = 4 * t + kq;
    xoff[t] = (uint32_t)(min(row, M - 1 - m0) * d * 2 + 16 * (r ^ (row & 15)));
  }
#pragma unroll
  for (int j = 0; j < TC; ++j) {
    const int row = lane >> 2;
    woff[j] = (uint32_t)(min(16 * (j % CT) + row, rows - 1) * (d >> 1) + 16 * ((lane & 3) ^ (row >> 2)));
  }
  const uint32_t one = fp16_1024_pair();
  f4 acc[4][4];
#pragma unroll
  for (int j = 0; j < TC; ++j)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[j][t] = f4{0.f, 0.f, 0.f, 0.f};

  // Scales and zeros of a chunk: lane 16 j + r fetches those of row r of tile j
  // and passes them on (fetched by every lane that uses them, one instruction
  // per tile, they cost more than the codes: 4096 -> 4096 at 32 tokens 9.7
  // against 8.0 us, 128 tokens 16.9 against 13.6). Groups of 64: both groups of
  // the chunk.
  const int js = kq % TC;
  const size_t srow = ((size_t)min(16 * (js % CT) + r, rows - 1) + c0 + (size_t)(js / CT) * N) * sgr;
  uint8_t* xl = lds + w * WB;
  uint8_t* wl = xl + 4096 * TT;

  for (int c = w; c < segs; c += nw) {
    const int gi = (128 * c) >> (6 + gsh);
    uint32_t sz0 = sc[srow + gi] | (uint32_t)zr[srow + gi] << 16, sz1 = 0;
    if (gsh == 0) sz1 = sc[srow + gi + 1] | (uint32_t)zr[srow + gi + 1] << 16;
#pragma unroll
    for (int j = 0; j < TC; ++j) {
      const __amdgpu_buffer_rsrc_t rw = codes(j / CT);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(wl + 1024 * j), 16, woff[j], 64 * c, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < 4 * TT; ++t)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(xl + 1024 * t), 16, xoff[t], 256 * c, 0, 0);
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
    u4 v[TC];
    h2 ss[TC], zz[TC], zz64[TC];
#pragma unroll
    for (int j = 0; j < TC; ++j) {
      uint32_t sz = __shfl((int)sz0, 16 * j + r);
      if (gsh == 0) {
        const uint32_t second = __shfl((int)sz1, 16 * j + r);
        sz = kq >= 2 ? second : sz;
      }
      v[j] = *(const u4*)(wl + 1024 * j + 64 * r + 16 * (kq ^ (r >> 2)));
      ss[j] = splat2(__builtin_bit_cast(_Float16, (uint16_t)(sz & 0xffffu)));
      const float zf = (float)(sz >> 16);
      zz[j] = splat2((_Float16)(1024.0f + zf));
      zz64[j] = splat2((_Float16)(64.0f + zf));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h8 b[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) b[t] = *(const h8*)(xl + 4096 * t + 256 * r + 16 * ((4 * kq + i) ^ r));
#pragma unroll
      for (int j = 0; j < TC; ++j) {
        const h8 a = dequant8(v[j][i], zz[j], zz64[j], ss[j], one);
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[t], acc[j][t], 0, 0, 0);
      }
    }
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);  // its LDS reads, before the next chunk's DMA
  }

  // acc[j][t][e] = Z[token m0 + 16 t + r][row 16 j + 4 kq + e], each wavefront's
  // in its own region; added in wavefront order, tiles shared out
#pragma unroll
  for (int j = 0; j < TC; ++j)
#pragma unroll
    for (int t = 0; t < TT; ++t) *(f4*)(xl + 1024 * (j * TT + t) + 16 * lane) = acc[j][t];
  __syncthreads();
  for (int b = w; b < CT * TT; b += nw) {
    f4 z[GT ? 2 : 1];
#pragma unroll
    for (int u = 0; u < (GT ? 2 : 1); ++u) {
      const uint8_t* p = lds + 1024 * (b + u * CT * TT) + 16 * lane;
      z[u] = *(const f4*)p;
      for (int k = 1; k < nw; ++k) z[u] += *(const f4*)(p + k * WB);
    }
    const int m = m0 + 16 * (b % TT) + r, n = c0 + 16 * (b / TT) + 4 * kq;
    if (m < M && n < N) epi_lane<EPI>(z, m, n, N, bias, aux, act, erf, y);
  }
}

template <int EPI, int TT, int TC>
hipError_t launch(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                  const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
                  const W4Epilogue& ep, hipStream_t stream) {
  const int gsh = group == 64 ? 0 : group == 128 ? 1 : 2;
  constexpr int NC = epi_gated(EPI) ? 8 * TC : 16 * TC;
  const int mblk = (int)((M + 16 * TT - 1) / (16 * TT));
  const int blocks = (int)((N + NC - 1) / NC) * mblk, per = (blocks + 7) / 8;
  // as many wavefronts as give each the same number of chunks
  const int segs = (int)(d / 128);
  constexpr int most = tile_waves(TT, TC);
  const int rounds = (segs + most - 1) / most, nw = (segs + rounds - 1) / rounds;
  hipLaunchKernelGGL((w4_tiles_kernel<EPI, TT, TC>), dim3(8u * (unsigned)per), dim3(64 * nw), 0, stream, x, qweight,
                     scales, zeros, bias, y, (int)M, (int)N, (int)d, gsh, mblk, blocks, per, ep.aux, act_form(ep.act),
                     (int)(ep.act == PARO_ACT_GELU));
  return hipGetLastError();
}

// Tile shapes, and what a round of one workgroup per CU costs: the time per
// chunk of k in the same unit (0.028 us; 4096 -> 4096, tiles in one round: 8.0,
// 9.4, 12.1 and 16.5 us).
struct Shape {
  int tt, tc, cost;
};
constexpr Shape kShapes[] = {{1, 2, 12}, {2, 2, 15}, {2, 4, 21}, {4, 4, 30}};

// Index of the shape whose rounds cost least, and that cost.
int best_shape(int64_t M, int64_t P, int64_t* least) {
  int best = 0;
  int64_t best_cost = 0;
  for (int i = 0; i < 4; ++i) {
    const Shape& s = kShapes[i];
    const int64_t tiles = ((M + 16 * s.tt - 1) / (16 * s.tt)) * ((P + 16 * s.tc - 1) / (16 * s.tc));
    const int64_t n = (tiles + kCus - 1) / kCus;
    if (!i || n * s.cost < best_cost) {
      best = i;
      best_cost = n * s.cost;
    }
  }
  *least = best_cost;
  return best;
}

template <int EPI>
hipError_t launch_epi(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                      const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
                      const W4Epilogue& ep, hipStream_t stream) {
  int64_t cost;
  switch (best_shape(M, epi_gated(EPI) ? 2 * N : N, &cost)) {
    case 0: return launch<EPI, 1, 2>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
    case 1: return launch<EPI, 2, 2>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
    case 2: return launch<EPI, 2, 4>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
    default: return launch<EPI, 4, 4>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
  }
}

}  // namespace

// Against the kernels of w4_gemm_kernels.h: always at up to 64 tokens, and in
// one round of 64 x 64 tiles (1024 x 1024 at 333 tokens 10.4 against 6.5 us, ragged 2560
// -> 1040 14.8 against 9.6); up to 128 tokens in four (gated 4096 -> 14336 at 128
// tokens, four rounds, 105 against 65; 1024 -> 28672, seven, 41 against 49); from
// there on in three unless k is short (8192 -> 8192 at 333, three, 116 against
// 96; gated 4096 -> 4096 at 256, two, 36 against 38; gated 14336 -> 4096 at 333,
// three, 137 against 142; four and more lose: gated 8192 -> 8192 at 512 150
// against 225; 512 -> 8192 at 160, two, 10.7 against 13.1, the few chunks of a
// tile leaving most of a CU's wavefronts idle).
bool w4_tiles_fit(int64_t M, int64_t P, int64_t d) {
  if (M <= 64) return true;
  int64_t cost = 0;
  best_shape(M, P, &cost);
  const int64_t round = kShapes[3].cost;
  return cost <= round || (M <= 128 ? cost <= 4 * round : cost <= 3 * round && d >= 2048);
}

hipError_t launch_w4_tiles(int epi, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                           const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d,
                           int group, const W4Epilogue& ep, hipStream_t stream) {
  auto go = epi == kEpiAct        ? launch_epi<kEpiAct>
            : epi == kEpiGated    ? launch_epi<kEpiGated>
            : epi == kEpiActGrad ? launch_epi<kEpiActGrad>
                                 : launch_epi<kEpiGatedGrad>;
  return go(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
}

}  // namespace paro
