// gfx950 kernels for the gradient of a W4 product at its input,
//   dX'[m][k] = sum_p dZ[m][p] W_hat[p][k],
// W_hat[p][k] the fp16 number nearest to (q - z) s, P rows of weights.
// The contraction runs over the weight rows, along which neither the packed
// codes nor W_hat are contiguous, so W_hat^T [k][p] is written out first
// (dequantized and transposed through LDS, fp16, p padded with zeros to a
// multiple of 128) and the product is then a dense one of two operands whose
// contraction index is contiguous. W_hat^T costs 2.5 P d bytes moved whatever
// M is: 10.1 us for 4096 x 4096 (4.1 TB/s), 57 for 28672 x 4096 (5.2 TB/s, what
// a copy reaches), 15% of the product's time at 2048 tokens. The product itself
// is bound by the matrix cores under the power limit (busy 67% of the time at
// 2048 x 28672 -> 4096; 385 us at least, 400 on average over 20 calls from a
// cold clock, 1250 and 1200 TFLOP/s; a W4 operand dequantized on the way, 1120).
// dZ is the matrix cores' fp16 operand, as the caller gets it: dX' is off by
// 2.9e-4 of its norm against 64 bits, 2.1e-4 of which is its own rounding. The
// fp32 dZ as a sum of two fp16 terms would take the product twice.
#include <algorithm>
#include <type_traits>

#include "paro_internal.h"
#include "w4_common.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

using namespace w4;

constexpr int TP = 128, TD = 128;  // weight rows and channels per workgroup
constexpr int TS = TP / 2 + 4;     // LDS words per channel: two rows a word, rows 16-byte aligned

// wt[k][p] (row stride pp, a multiple of 128): 128 rows x 128 channels per
// workgroup. Lane l of wavefront w dequantizes rows 2 l and 2 l + 1, channels
// 32 w .. 32 w + 31 (16 bytes of each row, inside one group), and stores the
// pair of one channel as one word, so a wavefront's LDS store is 64
// consecutive words; channels then leave as runs of 256 bytes.
__global__ __launch_bounds__(256) void w4_transpose_kernel(const uint8_t* __restrict__ qw,
                                                           const uint16_t* __restrict__ sc,
                                                           const uint8_t* __restrict__ zr, int P, int d, int gsh,
                                                           uint16_t* __restrict__ wt, int pp) {
  __shared__ __attribute__((aligned(16))) uint32_t t[TD * TS];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int k0 = blockIdx.x * TD, p0 = blockIdx.y * TP;
  const int groups = d >> (6 + gsh);
  const int k = k0 + 32 * w;
  const uint32_t one = fp16_1024_pair();
  h8 v[2][4];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int p = p0 + 2 * lane + b;
    u4 c = {0u, 0u, 0u, 0u};
    uint16_t s = 0;
    float z = 0.0f;
    if (p < P) {  // (rows past P: scale zero, so zeros)
      c = *(const u4*)(qw + (size_t)p * (d >> 1) + (k >> 1));
      const size_t gi = (size_t)p * groups + (k >> (6 + gsh));
      s = sc[gi];
      z = (float)zr[gi];
    }
    const h2 ss = splat2(__builtin_bit_cast(_Float16, s));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[b][i] = dequant8(c[i], splat2((_Float16)(1024.0f + z)), splat2((_Float16)(64.0f + z)), ss, one);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u4 a = __builtin_bit_cast(u4, v[0][i]), b = __builtin_bit_cast(u4, v[1][i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // channels 8 i + 2 e and + 1 of the two rows
      t[(32 * w + 8 * i + 2 * e) * TS + lane] = (a[e] & 0xffffu) | (b[e] << 16);
      t[(32 * w + 8 * i + 2 * e + 1) * TS + lane] = (a[e] >> 16) | (b[e] & 0xffff0000u);
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < TD / 16; ++r) {
    const int kk = 16 * r + (tid >> 4), c = tid & 15;  // channel, chunk of 8 rows
    *(u4*)(wt + (size_t)(k0 + kk) * pp + p0 + 8 * c) = *(const u4*)&t[kk * TS + 4 * c];
  }
}

// out [M][pp] = in [M][P] with zeros in columns P .. pp - 1 (both multiples of 8)
__global__ __launch_bounds__(256) void pad_rows_kernel(const u4* __restrict__ in, int64_t M, int P8,
                                                       u4* __restrict__ out, int pp8) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * pp8; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / pp8;
    const int c = (int)(i - m * pp8);
    out[i] = c < P8 ? in[m * P8 + c] : u4{0u, 0u, 0u, 0u};
  }
}

// --------------------------------------------------------------------------
// The product dx[m][n] = sum_p dz[m][p] wt[n][p] (n the input channels), fp32
// sums, on v_mfma_f32_32x32x16_f16 with wt as the first operand, so that a lane
// holds four consecutive n of one m. Four wavefronts, one per SIMD; NWN of them
// along n, each TN x TM accumulator tiles of 32 x 32:
//   <4, 4, 2>  256 (n) x 256 (m) per workgroup: 8 operand reads per 16 MFMAs;
//   <4, 2, 2>  256 (n) x 128 (m);
//   <2, 2, 4>  256 (n) x 64 (m), for few tokens.
// k-tiles of 64 of both operands go straight from global memory into LDS
// (16-byte load-to-LDS DMA; row r keeps its chunk c at c ^ ((r >> 1) & 7), which
// spreads the 16 rows of an operand read over all 16-byte positions), wt into a
// ring of three stages, dz into one of two. While the MFMAs of a 16-wide step
// run, the wavefront reads the next step's operands; after step 2 of k-tile kt
// it waits for the operands of kt + 1 and the barrier, and step 3 reads the
// first of them. Nobody reads the stages of kt any more then: step 3 sends dz
// of kt + 2, and steps 0 and 1 of the next k-tile wt of kt + 3. The loads take
// the CU's path of 64 bytes a cycle for half of the MFMAs' time; all in step 3,
// as two stages of each operand would have it, they hold it for twice its
// length (matrix cores busy 48%), and k-tiles of 32 in four stages read half
// lines (59%, at a lower clock for the doubled L2 requests).
// k may be split over ksplit workgroups of one tile (consecutive slots of one
// XCD): the workgroups leave fp32 partial tiles in the workspace and the last
// to arrive adds them in split order.
// --------------------------------------------------------------------------
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int IG_N = 256, IG_K = 64;  // channels per workgroup, k-tile
constexpr int kRsrcWord3 = 0x00020000;  // gfx9 buffer resource word 3
constexpr int kWaitVmLgkm0 = 0x70;      // s_waitcnt vmcnt(0) lgkmcnt(0)
constexpr int kAuxL2R = 1;              // sc0: skip the per-CU cache
constexpr int kAuxSys = 17;             // sc0 | sc1: memory-side coherence

template <int TN, int TM, int NWN, bool SPLIT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1)))
void input_grad_kernel(const uint16_t* __restrict__ wt, const uint16_t* __restrict__ dz, int M, int N, int pp,
                       int mblk, int nblk, int per, int ksplit, uint16_t* __restrict__ dx, float* __restrict__ part,
                       uint32_t* __restrict__ cnt, int sys) {
  constexpr int BM = 32 * TM * (4 / NWN);     // tokens per workgroup
  static_assert(32 * TN * NWN == IG_N, "256 channels per workgroup");
  constexpr int CA = IG_N / 32, CB = BM / 32;  // load-to-LDS instructions per lane and k-tile
  constexpr int NF = TN * TM;                  // MFMAs per step
  __shared__ __attribute__((aligned(1024))) _Float16 A0[IG_N * IG_K], A1[IG_N * IG_K], A2[IG_N * IG_K];
  __shared__ __attribute__((aligned(1024))) _Float16 B0[BM * IG_K], B1[BM * IG_K];
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, g = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = w % NWN, wm = w / NWN;
  // workgroup b runs on XCD b % 8; each XCD takes `per` consecutive tiles of
  // the order with m fastest, so that its workgroups share few n-blocks
  const int xcd = blockIdx.x & 7, idx0 = blockIdx.x >> 3;
  const int ks = SPLIT ? idx0 % ksplit : 0, idx = SPLIT ? idx0 / ksplit : idx0;
  const int tile = xcd * per + idx;
  if (tile >= mblk * nblk) return;
  const int nb = tile / mblk, mb = tile - nb * mblk;
  const int n0 = nb * IG_N, m0 = mb * BM;
  const int H = pp / (2 * IG_K);  // pairs of k-tiles
  const int kt0 = SPLIT ? 2 * (int)((int64_t)ks * H / ksplit) : 0;
  const int KT = (SPLIT ? 2 * (int)((int64_t)(ks + 1) * H / ksplit) : 2 * H) - kt0;

  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(wt + (size_t)n0 * pp), (short)0, min(N - n0, IG_N) * pp * 2, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(dz + (size_t)m0 * pp), (short)0, min(M - m0, BM) * pp * 2, kRsrcWord3);
  // DMA c of wavefront w fills rows 8 (C w + c) .. + 7 (C of them per
  // wavefront); rows past the end repeat the last one (never stored)
  uint32_t aoff[8], boff[8];
#pragma unroll
  for (int c = 0; c < CA; ++c) {
    const int r = 8 * (CA * w + c) + (lane >> 3);
    aoff[c] = (uint32_t)(min(r, N - 1 - n0) * pp + 8 * ((lane & 7) ^ ((r >> 1) & 7))) * 2u;
  }
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const int r = 8 * (CB * w + c) + (lane >> 3);
    boff[c] = (uint32_t)(min(r, M - 1 - m0) * pp + 8 * ((lane & 7) ^ ((r >> 1) & 7))) * 2u;
  }
  // (past the last k-tile: the last one again, into a stage nobody reads)
  auto dma_a = [&](int kt, int half, _Float16* as) {  // in two halves
    const int k = (kt0 + min(kt, KT - 1)) * IG_K * 2;
#pragma unroll
    for (int c = CA / 2 * half; c < CA / 2 * (half + 1); ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)&as[(CA * w + c) * 512], 16, aoff[c], k, 0, 0);
  };
  auto dma_b = [&](int kt, _Float16* bs) {
    const int k = (kt0 + min(kt, KT - 1)) * IG_K * 2;
#pragma unroll
    for (int c = 0; c < CB; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)&bs[(CB * w + c) * 512], 16, boff[c], k, 0, 0);
  };
  f16v acc[4][4];
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[j][i][e] = 0.0f;
  // operands of step s of a k-tile: lane half g takes chunk 4 g + s of each row
  auto read = [&](const _Float16* as, const _Float16* bs, int s, h8* a, h8* b) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int r = 32 * (TN * wn + j) + l32;
      a[j] = *(const h8*)(as + r * IG_K + 8 * ((4 * g + s) ^ ((r >> 1) & 7)));
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = 32 * (TM * wm + i) + l32;
      b[i] = *(const h8*)(bs + r * IG_K + 8 * ((4 * g + s) ^ ((r >> 1) & 7)));
    }
  };
  // one step: its MFMAs on the operands in hand, behind the next step's reads,
  // with NL loads spread among them
  h8 a[4], b[4], an[4], bn[4];
  auto step = [&](auto loads) {
    constexpr int NL = decltype(loads)::value, PER = NL == 0 || NF < NL ? 1 : NF / (NL == 0 ? 1 : NL);
#pragma unroll
    for (int f = 0; f < NF; ++f)
      acc[f / TM][f % TM] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[f / TM], b[f % TM], acc[f / TM][f % TM], 0, 0, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, TN + TM, 0);
#pragma unroll
    for (int c = 0; c < NL; ++c) {
      __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
      __builtin_amdgcn_sched_group_barrier(0x004, 1, 0);  // the load's M0 write
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t < TN) a[t] = an[t];
      if (t < TM) b[t] = bn[t];
    }
  };
  // s_waitcnt with lgkmcnt(0) and vmcnt(v): at most v loads still on their way
  constexpr auto wait_vm = [](int v) { return 0x70 | (v & 15) | ((v >> 4) << 14); };
  // k-tile kt in (as, bs), kt + 1 in (as1, bs1); ap: the wt stage of kt - 1,
  // which kt + 2 takes
  auto ktile = [&](int kt, _Float16* ap, const _Float16* as, _Float16* bs, const _Float16* as1, const _Float16* bs1) {
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      if (s < 2) dma_a(kt + 2, s, ap);
      read(as, bs, s + 1, an, bn);
      if (s < 2) step(std::integral_constant<int, CA / 2>{});
      else step(std::integral_constant<int, 0>{});
    }
    // still on their way: wt of kt + 2
    __builtin_amdgcn_s_waitcnt(wait_vm(CA));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    dma_b(kt + 2, bs);
    read(as1, bs1, 0, an, bn);
    step(std::integral_constant<int, CB>{});
  };

  dma_a(0, 0, A0);
  dma_a(0, 1, A0);
  dma_b(0, B0);
  dma_a(1, 0, A1);
  dma_a(1, 1, A1);
  dma_b(1, B1);
  __builtin_amdgcn_s_waitcnt(wait_vm(CA + CB));
  __builtin_amdgcn_s_barrier();
  read(A0, B0, 0, a, b);
  int kt = 0;
  for (; kt + 6 <= KT; kt += 6) {  // both rings' periods; KT is even (p is padded to pairs)
    ktile(kt, A2, A0, B0, A1, B1);
    ktile(kt + 1, A0, A1, B1, A2, B0);
    ktile(kt + 2, A1, A2, B0, A0, B1);
    ktile(kt + 3, A2, A0, B1, A1, B0);
    ktile(kt + 4, A0, A1, B0, A2, B1);
    ktile(kt + 5, A1, A2, B1, A0, B0);
  }
  if (kt < KT) {
    ktile(kt, A2, A0, B0, A1, B1);
    ktile(kt + 1, A0, A1, B1, A2, B0);
  }
  if (kt + 2 < KT) {
    ktile(kt + 2, A1, A2, B0, A0, B1);
    ktile(kt + 3, A2, A0, B1, A1, B0);
  }
  __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);  // the last DMA writes a stage that is used below
  __builtin_amdgcn_s_barrier();

  if constexpr (SPLIT) {
    auto rsrc = [&](int k2) {
      return __builtin_amdgcn_make_buffer_rsrc((void*)(part + ((size_t)tile * ksplit + k2) * (size_t)(IG_N * BM)),
                                               (short)0, IG_N * BM * 4, kRsrcWord3);
    };
    const __amdgpu_buffer_rsrc_t rmine = rsrc(ks);
#pragma unroll
    for (int f = 0; f < 4 * NF; ++f) {
      const int j = f / (4 * TM), i = f / 4 % TM, q = f % 4;
      const u4 v = __builtin_bit_cast(u4, f4{acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2],
                                             acc[j][i][4 * q + 3]});
      const int off = ((w * 4 * NF + f) * 64 + lane) * 16;
      if (sys) __builtin_amdgcn_raw_buffer_store_b128(v, rmine, off, 0, kAuxSys);
      else __builtin_amdgcn_raw_buffer_store_b128(v, rmine, off, 0, 0);
    }
    // (the stages take all of LDS; the epilogue uses A0)
    if (!arrive_last(&cnt[tile], ksplit, sys, (uint32_t*)B0)) return;
    // With two pieces the last keeps its own sums in registers and reads the
    // other's; the 256 x 256 tile's 256 accumulators would spill for it
    constexpr bool kKeep = NF < 16;
    auto load4 = [&](const __amdgpu_buffer_rsrc_t rk, int f) {
      const int off = ((w * 4 * NF + f) * 64 + lane) * 16;
      return __builtin_bit_cast(f4, sys ? __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, kAuxSys)
                                        : __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, kAuxL2R));
    };
    if (kKeep && ksplit == 2) {  // one sum, the same in either order
      const __amdgpu_buffer_rsrc_t rk = rsrc(1 - ks);
#pragma unroll
      for (int f0 = 0; f0 < 4 * NF; f0 += 8) {
        f4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = load4(rk, f0 + e);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int f = f0 + e, j = f / (4 * TM), i = f / 4 % TM, q = f % 4;
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[j][i][4 * q + c] += v[e][c];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int f0 = 0; f0 < 4 * NF; f0 += 16) {
        f4 r[16];
        for (int k2 = 0; k2 < ksplit; ++k2) {
          const __amdgpu_buffer_rsrc_t rk = rsrc(k2);
          f4 v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = load4(rk, f0 + e);
#pragma unroll
          for (int e = 0; e < 16; ++e) r[e] = k2 == 0 ? v[e] : r[e] + v[e];
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int f = f0 + e, j = f / (4 * TM), i = f / 4 % TM, q = f % 4;
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[j][i][4 * q + c] = r[e][c];
        }
      }
    }
  }

  // acc[j][i][e] = dx[n = nw + 32 j + 8 (e / 4) + 4 g + e % 4][m = mw + 32 i + l32],
  // out through 8 KB of LDS per wavefront in blocks of 64 x 64, whole 128-byte rows
  const int nw = n0 + 32 * TN * wn, mw = m0 + 32 * TM * wm;
  uint8_t* stage = (uint8_t*)A0 + 8192 * w;
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int jh = 0; jh < TN / 2; ++jh) {
#pragma unroll
    for (int ih = 0; ih < TM / 2; ++ih) {
#pragma unroll
      for (int jj = 0; jj < 2; ++jj)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const f16v& v = acc[2 * jh + jj][2 * ih + t];
            const int nl = 32 * jj + 8 * q + 4 * g, rl = 32 * t + l32;
            *(u2*)(stage + rl * 128 + (((nl >> 3) ^ (rl & 7)) << 4) + (((nl >> 2) & 1) << 3)) =
                u2{half_bits(v[4 * q]) | (half_bits(v[4 * q + 1]) << 16),
                   half_bits(v[4 * q + 2]) | (half_bits(v[4 * q + 3]) << 16)};
          }
#pragma unroll
      for (int rr = 0; rr < 8; ++rr) {
        const int rl = 8 * rr + (lane >> 3), c = lane & 7;
        const u4 v = *(const u4*)(stage + rl * 128 + ((c ^ (rl & 7)) << 4));
        const int m = mw + 64 * ih + rl, n = nw + 64 * jh + 8 * c;
        if (m < M && n < N) *(u4*)(dx + (size_t)m * N + n) = v;
      }
    }
  }
}

size_t a256(size_t b) { return (b + 255) & ~(size_t)255; }
int64_t pad128(int64_t n) { return (n + 127) & ~int64_t(127); }

// Tile and k split of the product: the least estimated time, in k-tiles of the
// 256 x 256 tile, over the tile heights and splits: 6 for a round's start and
// end, and for a split's meeting 5 and 4 per piece of 256 tokens (with the
// transposition, 1024 tokens x 4096 -> 4096 in 256 tiles of 64 53 us, in 128 of
// 128 and two pieces 57; 1024 x 14336 -> 4096 172 and 205).
struct GradPlan {
  int bm = 256, ksplit = 1;
  int64_t mblk = 0, nblk = 0, tiles = 0;
  size_t partial_bytes = 0;
};
GradPlan plan_input_grad(int64_t M, int64_t P, int64_t d) {
  GradPlan best;
  double best_cost = 0;
  const int64_t H = pad128(P) / (2 * IG_K);
  for (int bm : {256, 128, 64}) {
    GradPlan p;
    p.bm = bm;
    p.mblk = (M + bm - 1) / bm;
    p.nblk = (d + IG_N - 1) / IG_N;
    p.tiles = p.mblk * p.nblk;
    const double kt = bm == 256 ? 1.0 : bm == 128 ? 0.6 : 0.4;  // a k-tile's time
    for (int ks = 1; ks <= 16 && ks <= H; ks *= 2) {
      if (ks > 1 && (p.tiles > (int64_t)(kDecodeCounterBytes / 4) || p.tiles * ks > 512)) break;
      const int64_t rounds = (8 * ((p.tiles + 7) / 8) * ks + 255) / 256;
      const int64_t len = 2 * ((H + ks - 1) / ks);
      const double cost = rounds * (len * kt + 6) + (ks > 1 ? 5 + (bm / 256.0) * 4 * ks : 0);
      if (best.mblk == 0 || cost < best_cost) {
        best = p;
        best.ksplit = ks;
        best_cost = cost;
      }
    }
  }
  if (best.ksplit > 1) best.partial_bytes = (size_t)best.tiles * best.ksplit * IG_N * best.bm * 4;
  return best;
}

template <int TN, int TM, int NWN>
void launch_tiles(const GradPlan& p, const uint16_t* wt, const uint16_t* dz, int M, int N, int pp, uint16_t* dx,
                  float* part, uint32_t* cnt, hipStream_t stream) {
  const int per = (int)((p.tiles + 7) / 8);
  const dim3 grid(8u * (unsigned)per * (unsigned)p.ksplit);
  if (p.ksplit > 1)
    hipLaunchKernelGGL((input_grad_kernel<TN, TM, NWN, true>), grid, dim3(256), 0, stream, wt, dz, M, N, pp,
                       (int)p.mblk, (int)p.nblk, per, p.ksplit, dx, part, cnt, (int)!xcd_dispatch_is_round_robin());
  else
    hipLaunchKernelGGL((input_grad_kernel<TN, TM, NWN, false>), grid, dim3(256), 0, stream, wt, dz, M, N, pp,
                       (int)p.mblk, (int)p.nblk, per, 1, dx, nullptr, nullptr, 0);
}

}  // namespace

size_t input_grad_scratch_bytes(int64_t M, int64_t P, int64_t d) {
  if (input_grad_rows_fit(M)) return a256(input_grad_rows_bytes(M, P, d));
  const int64_t pp = pad128(P);
  return a256((size_t)d * pp * 2) + (pp != P ? a256((size_t)M * pp * 2) : 0) + plan_input_grad(M, P, d).partial_bytes;
}

hipError_t launch_w4_input_grad(const uint16_t* dz, const uint8_t* qweight, const uint16_t* scales,
                                const uint8_t* zeros, uint16_t* dx, int64_t M, int64_t P, int64_t d, int group,
                                uint32_t* cnt, void* ws, hipStream_t stream) {
  if (input_grad_rows_fit(M))
    return launch_w4_input_grad_rows(dz, qweight, scales, zeros, dx, M, P, d, group, ws, stream);
  const int gsh = group == 64 ? 0 : group == 128 ? 1 : 2;
  const int64_t pp = pad128(P);
  char* at = (char*)ws;
  uint16_t* wt = (uint16_t*)at;
  at += a256((size_t)d * pp * 2);
  const dim3 grid((unsigned)(d / TD), (unsigned)(pp / TP));
  hipLaunchKernelGGL(w4_transpose_kernel, grid, dim3(256), 0, stream, qweight, scales, zeros, (int)P, (int)d, gsh, wt,
                     (int)pp);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (pp != P) {  // the product reads whole k-tiles, and no row may read its neighbour
    uint16_t* padded = (uint16_t*)at;
    at += a256((size_t)M * pp * 2);
    const int64_t blocks = (M * (pp / 8) + 255) / 256;
    hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)std::min<int64_t>(blocks, 16384)), dim3(256), 0, stream,
                       (const u4*)dz, M, (int)(P / 8), (u4*)padded, (int)(pp / 8));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    dz = padded;
  }
  const GradPlan p = plan_input_grad(M, P, d);
  auto go = p.bm == 256 ? launch_tiles<4, 4, 2> : p.bm == 128 ? launch_tiles<4, 2, 2> : launch_tiles<2, 2, 4>;
  go(p, wt, dz, (int)M, (int)d, (int)pp, dx, (float*)at, cnt, stream);
  return hipGetLastError();
}

}  // namespace paro
