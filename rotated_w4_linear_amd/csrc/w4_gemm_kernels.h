// gfx950 kernels for the W4G128 linear layer on rotated activations with
// many tokens (prefill, M > 16):
//   Y[m][n] = sum_k X'[m][k] (q[n][k] - z[n][k/G]) s[n][k/G] + b[n]
// (CSDN article section 2.1: Y = (X T^-1)(T W) + b; paper notes "主实验":
// 4-bit weights, group G = 128; 64 and 256 are taken as well, each 64-channel
// k-tile reading the one group it lies in). Here the layer is a dense contraction and runs
// on the matrix cores. Dequantization (w4_common.h): two codes at a time are
// masked into the mantissas of a pair of fp16 1024.0 values with one
// v_and_or_b32, (1024 + q) - (1024 + z) = q - z is exact in packed fp16, and
// one packed multiply by the fp16 scale rounds once.
#pragma once

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

// --------------------------------------------------------------------------
// prefill (M > 16): MFMA v_mfma_f32_32x32x16_f16 with the dequantized weights
// as operand A (32 output channels x 16 k) and X' as operand B (16 k x 32
// tokens). A wavefront owns a 64 (n) x 128 (m) tile: 2 x 4 accumulator tiles,
// 128 fp32 per lane, so two wavefronts fit on a SIMD and one's dequantization
// overlaps the other's MFMAs. A group of four wavefronts shares a 128 (m) x
// 256 (n) workgroup tile.
//
// Staging: every operand of a k-tile of 64 (X' tile, packed codes, the
// tile's group scale and zero of each row) goes from global memory straight
// into LDS with load-to-LDS DMA (16 bytes per lane for X' and codes), into
// two stages: the DMA of k-tile kt + 1 runs while k-tile kt is multiplied,
// and nothing is staged through registers. Each stage is its own LDS object,
// so the compiler sees that the stage being filled never aliases the one
// being read; the kernel waits for the DMA counter itself (s_waitcnt) before
// the one barrier per k-tile.
//  * X' tile [128 rows][8 chunks of 8 halfs]; chunk c of row r stored at
//    position c ^ ((r >> 1) & 7);
//  * packed int4 weight tile [256 rows][2 halves of 16 bytes]; half h of row r
//    at position h ^ ((r >> 3) & 1).
// A gfx950 16-byte LDS read is conflict-free when every 16 consecutive lanes
// address positions distinct modulo 16: the operand reads take 16 consecutive
// rows at a fixed chunk, which these swizzles spread over all 16 positions.
// DMA writes land lane-contiguously, so the swizzle is applied by choosing
// which source chunk each lane fetches. Each wavefront dequantizes its own 64
// rows in registers.
// With KS = 2 two groups of four wavefronts split k in halves inside the
// workgroup (for layers with few output tiles) and add their accumulators
// through LDS at the end.
//
// k order inside an MFMA: for a 64-wide k-tile, lane l (row n = l % 32,
// half g = l / 32) takes the codes 32 g .. 32 g + 31 of its row; MFMA step
// i (0..3) uses codes 32 g + 8 i .. + 7, so the four steps together contract
// k = 8 i + {0..7, 32..39}, and X' is read with the same mapping.
// --------------------------------------------------------------------------
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int GB_N = 256, GB_K = 64;
constexpr int GB_WSTAGE = GB_N * 2;     // 16-byte chunks per weight stage (8 KB)
constexpr int kRsrcWord3 = 0x00020000;  // gfx9 buffer resource word 3
// buffer access cache bits: sc0 (skip the per-CU cache) for loads of data
// another workgroup stored; sc0 | sc1 (memory-side) where workgroups may sit
// on different XCDs
constexpr int kAuxL2R = 1;
constexpr int kAuxSysW = 17;
// s_waitcnt immediate (gfx9 encoding): vmcnt(0) lgkmcnt(0), expcnt untouched
constexpr int kWaitVmLgkm0 = 0x70;
// vmcnt(8) lgkmcnt(0)
constexpr int kWaitVm8Lgkm0 = 0x78;
// vmcnt(4) lgkmcnt(0)
constexpr int kWaitVm4Lgkm0 = 0x74;
// lgkmcnt(0) alone (vmcnt and expcnt at their maxima)
constexpr int kWaitLgkm0 = 0xC07F;
// Output tiles (at 128 tokens) below which 64-token tiles are used: measured
// on MI355X, 64-token tiles win at 128 tiles (1024 x 4096 -> 4096: 699
// against 581 TFLOP/s) and lose at 256 (2048 x 4096 -> 4096: 760 against 918).
constexpr int64_t kHalfTileBelow = 256;
// 64-token tiles below which the tiles are also narrowed to 128 channels, so
// that every CU gets a workgroup
constexpr int64_t kNarrowTileBelow = 256;
// k-tiles per group of wavefronts below which the 64 x 128-tile kernel does
// not split k further across workgroups
constexpr int64_t kMinNarrowSplitKT = 4;
// 256 x 256 tiles (at 256 tokens) from which the wide kernel is used: measured
// on MI355X, 4096 x 4096 -> 4096 (256 tiles): 128 against 135 us; 2048 x
// 14336 -> 4096 (128 tiles) runs 372 against 288 us
constexpr int64_t kWideMinTiles = 256;
// Stream-K (the wide kernel with the tiles' k-tiles shared out evenly among
// the workgroups of each XCD) when each workgroup's range holds at least
// kMinSplitKT k-tiles: the partial tiles (256 KB per piece, written and read
// back) pay off only on long ranges. Measured on MI355X with uniform splits:
// 2048 x 14336 -> 4096 (two splits of 112 k-tiles) 242 against 292 us for the
// 128 x 256-tile kernel; 2048 x 4096 -> 4096 (two of 32) 88 against 73 us,
// 2048 x 4096 -> 1024 (eight of 8) 102 against 48 us
constexpr int64_t kMinSplitKT = 48;
// k-tiles a stream-K range is charged for cutting tiles at unequal k (see
// plan_w4_gemm)
constexpr int64_t kSkMisaligned = 20;
// n tiles of 32 channels per wavefront in the wide kernel
constexpr int kWideWN = 2;

// Tile row r of the weight block whose first output channel is nw0, as a row
// relative to row nw0 of the packed weights (rows past N repeat the last one).
// Gated: runs of eight gate rows, then the eight up rows of the same channels.
template <bool GT>
__device__ __forceinline__ int weight_row(int r, int N, int nw0) {
  if constexpr (!GT) return min(r, N - 1 - nw0);
  return min(8 * (r >> 4) + (r & 7), N - 1 - nw0) + ((r >> 3) & 1) * N;
}
// Packed rows from nw0 on that a tile of gn rows may touch (its up rows lie N
// rows further on).
template <bool GT>
__device__ __forceinline__ int weight_rows(int N, int nw0, int gn) {
  return GT ? N + min(N - nw0, gn / 2) : min(N - nw0, gn);
}

// MT: 32-token m tiles per wavefront (4: 128-token workgroup tiles; 2: 64,
// for layers with few output tiles). NT: 32-channel n tiles per wavefront (2:
// 256-channel workgroup tiles; 1: 128, for layers with fewer still). SPLIT: k
// also split across ksplit workgroups per tile (consecutive slots of one
// XCD), which meet through fp32 partial tiles; the last to arrive adds them
// in split order. EPI: the epilogue (w4_epilogue.h). For the gated ones N is
// the number of output channels, the weight block has 2 N rows (gate, then
// up) and a tile of GN rows takes GN / 2 channels, gate and up rows in runs of
// eight: an accumulator tile then holds both halves of its channels in the
// same lane, and the product of the halves needs no exchange.
template <int KS, int MT, int NT, bool SPLIT, int EPI>
__global__ __launch_bounds__(256 * KS) __attribute__((amdgpu_waves_per_eu(2)))
void w4_gemm_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ qw,
                    const uint16_t* __restrict__ sc, const uint8_t* __restrict__ zr,
                    const uint16_t* __restrict__ bias, uint16_t* y, int M, int N,
                    int d, int gsh, int mblk, int nblk, int ksplit, float* __restrict__ part,
                    uint32_t* __restrict__ cnt, int sys, int mmaj, const uint16_t* aux, ActForm act, int erf) {
  constexpr bool GT = epi_gated(EPI);
  constexpr int GB_M = 32 * MT;           // tokens per workgroup tile
  constexpr int GN = 128 * NT;            // output channels per workgroup tile
  constexpr int GB_XSTAGE = GB_M * GB_K;  // halfs per X' stage (16 KB at MT = 4)
  __shared__ __attribute__((aligned(1024))) _Float16 X0[KS][GB_XSTAGE], X1[KS][GB_XSTAGE];
  __shared__ __attribute__((aligned(1024))) u4 W0[KS][GB_WSTAGE], W1[KS][GB_WSTAGE];
  __shared__ __attribute__((aligned(16))) uint32_t S0[KS][GB_N], S1[KS][GB_N];
  __shared__ __attribute__((aligned(16))) uint32_t Z0[KS][GB_N], Z1[KS][GB_N];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int kg = __builtin_amdgcn_readfirstlane(tid >> 8);     // k group (KS > 1)
  const int w = __builtin_amdgcn_readfirstlane((tid >> 6) & 3);  // wavefront inside the group
  // XCD-aware tile order: workgroup b runs on XCD b % 8. XCD x owns the
  // n-blocks x, x + 8, ... and walks them in super-blocks of 8 m-blocks x all
  // its n-blocks, so the workgroups resident on one XCD share both their X'
  // and their weight k-tiles through its L2; or (mmaj, layers with a large X'
  // and N < 4 M) XCD x owns the m-blocks x, x + 8, ... and all n-blocks, so
  // that it reads only its eighth of X'.
  const int xcd = blockIdx.x & 7, idx0 = blockIdx.x >> 3;
  if (!SPLIT) ksplit = 1;
  const int ks = idx0 % ksplit, idx = idx0 / ksplit;
  int mb, nb;
  if (mmaj) {
    // XCD x owns the m-blocks x, x + 8, ... and all n-blocks of each
    const int mi = idx / nblk;
    mb = xcd + 8 * mi;
    nb = idx - mi * nblk;
    if (mb >= mblk) return;
  } else {
    const int nbx = (nblk - xcd + 7) >> 3;
    if (nbx <= 0) return;
    const int mg = idx / (8 * nbx), rem = idx - mg * 8 * nbx;
    nb = xcd + 8 * (rem / 8);
    mb = mg * 8 + (rem & 7);
    if (mb >= mblk) return;
  }
  const int m0 = mb * GB_M;
  const int nw0 = nb * (GT ? GN / 2 : GN);            // workgroup's first output channel
  const int n0 = nw0 + (GT ? 16 : 32) * NT * w;       // this wavefront's first output channel
  const int groups = d >> (6 + gsh);  // quantization groups of 64 << gsh channels per row
  const int KT = (d / GB_K) / (KS * ksplit);  // k-tiles per group of wavefronts
  const int kt0 = (ks * KS + kg) * KT;
  const int l32 = lane & 31, g = lane >> 5;

  // Buffer resources based at this tile's first row (byte offsets < 2^31,
  // checked on the host); rows past M or N are clamped to the last row.
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(x + (size_t)m0 * d), (short)0, min(M - m0, GB_M) * d * 2, kRsrcWord3);
  const int wrows = weight_rows<GT>(N, nw0, GN);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(qw + (size_t)nw0 * (d >> 1)), (short)0, wrows * (d >> 1), kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(sc + (size_t)nw0 * groups), (short)0, wrows * groups * 2, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rz = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(zr + (size_t)nw0 * groups), (short)0, wrows * groups, kRsrcWord3);
  // X' DMA c of wavefront w fills tile rows 8 (MT w + c) .. + 7; the lane at
  // position l % 8 of row l / 8 fetches the source chunk (l % 8) ^ swizzle
  // (arrays the lambdas below capture are sized for MT = 4: the host pass of
  // hipcc cannot instantiate lambdas capturing arrays of template-dependent
  // size)
  uint32_t xoff[4];
#pragma unroll
  for (int c = 0; c < MT; ++c) {
    const int r = 8 * (MT * w + c) + (lane >> 3);
    const int row = min(r, M - 1 - m0);
    xoff[c] = (uint32_t)(row * d + 8 * ((lane & 7) ^ ((r >> 1) & 7))) * 2u;
  }
  // code DMA c of wavefront w fills tile rows 32 (NT w + c) .. + 31
  uint32_t woff[2];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const int r = 32 * (NT * w + c) + (lane >> 1);
    const int row = weight_row<GT>(r, N, nw0);
    woff[c] = (uint32_t)(row * (d >> 1) + 16 * ((lane & 1) ^ ((r >> 3) & 1)));
  }
  // group scale and zero: lane l of wavefront w fetches row 64 w + l (NT = 1:
  // wavefronts 0 and 1 fetch the 128 rows)
  const bool szw = NT == 2 || w < 2;
  const uint32_t szrow = (uint32_t)(weight_row<GT>(64 * w + lane, N, nw0) * groups);

  // the DMA of one k-tile: MT + NT + 2 load-to-LDS instructions per lane
  auto dma = [&](int kt, _Float16* xs, u4* ws, uint32_t* ss_l, uint32_t* zs_l) {
    const int kglob = kt0 + kt;
    const uint32_t gi = (uint32_t)(kglob >> gsh);  // the k-tile's group (64-channel k-tiles)
    if (szw) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)&ss_l[64 * w], 2, (szrow + gi) * 2u, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rz, (lds_void*)&zs_l[64 * w], 1, szrow + gi, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < MT; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)&xs[(MT * w + c) * 64 * 8], 16, xoff[c],
                                               kglob * GB_K * 2, 0, 0);
#pragma unroll
    for (int c = 0; c < NT; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)&ws[(NT * w + c) * 64], 16, woff[c],
                                               kglob * (GB_K / 2), 0, 0);
  };

  const uint32_t one = fp16_1024_pair();
  f16v acc[2][4];  // n tiles j < NT and m tiles mm < MT used
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int mm = 0; mm < MT; ++mm)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[j][mm][e] = 0.0f;

  // One k-tile from stage (xs, ws, ss_l, zs_l) while the DMA of the next
  // k-tile fills the other stage, then wait for that DMA and one barrier.
  // Past the last tile the DMA reloads the last tile into a stage nobody reads.
  auto step = [&](int kt, const _Float16* xb, const u4* wl, const uint32_t* ss_l,
                  const uint32_t* zs_l, _Float16* xn, u4* wn, uint32_t* sn, uint32_t* zn) {
    dma(min(kt + 1, KT - 1), xn, wn, sn, zn);
    __builtin_amdgcn_sched_barrier(0);
    u4 wf[2];
    h2 ss[2], zz[2], zz64[2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = 32 * NT * w + 32 * j + l32;
      wf[j] = wl[2 * r + (g ^ ((r >> 3) & 1))];
      // (rows past N read the last row's scale, clamped by the DMA; never stored)
      ss[j] = splat2(__builtin_bit_cast(_Float16, (uint16_t)(ss_l[r] & 0xffffu)));
      const float zf = (float)(zs_l[r] & 0xffu);
      zz[j] = splat2((_Float16)(1024.0f + zf));
      zz64[j] = splat2((_Float16)(64.0f + zf));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h8 a[2], b[MT];
#pragma unroll
      for (int j = 0; j < NT; ++j) a[j] = dequant8(wf[j][i], zz[j], zz64[j], ss[j], one);
#pragma unroll
      for (int mm = 0; mm < MT; ++mm) {
        const int r = 32 * mm + l32;
        b[mm] = *(const h8*)(xb + r * GB_K + 8 * ((4 * g + i) ^ ((r >> 1) & 7)));
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int mm = 0; mm < MT; ++mm)
          acc[j][mm] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[j], b[mm], acc[j][mm], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
    __builtin_amdgcn_s_barrier();
  };

  dma(0, &X0[kg][0], &W0[kg][0], &S0[kg][0], &Z0[kg][0]);
  __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
  __builtin_amdgcn_s_barrier();
  for (int kt = 0; kt < KT; kt += 2) {
    step(kt, &X0[kg][0], &W0[kg][0], &S0[kg][0], &Z0[kg][0], &X1[kg][0], &W1[kg][0], &S1[kg][0], &Z1[kg][0]);
    if (kt + 1 < KT) step(kt + 1, &X1[kg][0], &W1[kg][0], &S1[kg][0], &Z1[kg][0], &X0[kg][0], &W0[kg][0], &S0[kg][0], &Z0[kg][0]);
  }

  // the epilogue's second operand (read by the wavefronts of group 0), on its
  // way while the groups' sums meet
  u4 av[2][8];
  if constexpr (EPI != kEpiPlain) {
    if (kg == 0) {
#pragma unroll
      for (int ps = 0; ps < MT / 2; ++ps) epi_fetch<EPI, NT>(av[ps], lane, m0 + 64 * ps, n0, M, N, aux);
    }
  }
  if constexpr (KS > 1) {
    // the k groups add their partial sums pairwise through LDS, (0 + 1) +
    // (2 + 3): in the round of span s, group kg = r + s hands its sums to
    // group r (r a multiple of 2 s) through the X' stages 0 of groups r and
    // r + 1 (32 KB at MT = 4, 16 KB at MT = 2), PM m tiles of one n tile
    // (16 KB per m tile) at a time
    constexpr int PM = MT / 2;
#pragma unroll
    for (int span = 1; span < KS; span *= 2) {
      const int pos = kg & (2 * span - 1);
      float* red = (float*)&X0[kg - pos][0];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int h = 0; h < MT / PM; ++h) {
          if (pos == span) {
#pragma unroll
            for (int mm = 0; mm < PM; ++mm)
#pragma unroll
              for (int e = 0; e < 16; ++e) red[((w * PM + mm) * 16 + e) * 64 + lane] = acc[j][PM * h + mm][e];
          }
          __syncthreads();
          if (pos == 0) {
#pragma unroll
            for (int mm = 0; mm < PM; ++mm)
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[j][PM * h + mm][e] += red[((w * PM + mm) * 16 + e) * 64 + lane];
          }
          __syncthreads();
        }
      }
    }
    if constexpr (!SPLIT) {
      if (kg != 0) return;
    }
  }

  if constexpr (SPLIT) {
    // Split k across workgroups: group 0 of every workgroup of the tile stores
    // its fp32 partial tile ([w][f][lane] 16-byte chunks, GB_M x GN floats)
    // and the workgroup counts itself in; the last to arrive adds the partial
    // tiles in split order (so the sum does not depend on the order of
    // arrival), resets the counter and runs the epilogue. The workgroups of a
    // tile share an XCD: plain stores, an L2 atomic and loads that skip the
    // per-CU cache suffice; where the dispatch rule is not established (sys)
    // they go through memory. Every wavefront takes part in the barriers.
    __shared__ uint32_t s_last;
    const int tile = mb * nblk + nb;
    constexpr int NF = NT * MT * 4;  // 16-byte chunks per lane
    auto rsrc = [&](int k2) {
      return __builtin_amdgcn_make_buffer_rsrc(
          (void*)(part + ((size_t)tile * ksplit + k2) * (size_t)(GB_M * GN)), (short)0, GB_M * GN * 4, kRsrcWord3);
    };
    if (kg == 0) {
      const __amdgpu_buffer_rsrc_t rmine = rsrc(ks);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int j = f / (MT * 4), mm = (f / 4) % MT, q = f % 4;
        const u4 v = __builtin_bit_cast(u4, f4{acc[j][mm][4 * q], acc[j][mm][4 * q + 1], acc[j][mm][4 * q + 2],
                                               acc[j][mm][4 * q + 3]});
        const int off = ((w * NF + f) * 64 + lane) * 16;
        if (sys) __builtin_amdgcn_raw_buffer_store_b128(v, rmine, off, 0, kAuxSysW);
        else __builtin_amdgcn_raw_buffer_store_b128(v, rmine, off, 0, 0);
      }
    }
    __builtin_amdgcn_s_waitcnt(0);  // this wavefront's stores have reached L2 / memory
    __syncthreads();
    if (tid == 0) {
      uint32_t old;
      if (sys) old = __hip_atomic_fetch_add(&cnt[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
      else old = __hip_atomic_fetch_add(&cnt[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s_last = old == (uint32_t)(ksplit - 1);
    }
    __syncthreads();
    if (!s_last || kg != 0) return;
    // (all of a split's loads before the first sum: taken one at a time, their
    // way from L2 adds up)
    f4 t[NF];
    for (int k2 = 0; k2 < ksplit; ++k2) {
      const __amdgpu_buffer_rsrc_t rk = rsrc(k2);
      f4 v[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int off = ((w * NF + f) * 64 + lane) * 16;
        v[f] = __builtin_bit_cast(f4, sys ? __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, kAuxSysW)
                                          : __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, kAuxL2R));
      }
#pragma unroll
      for (int f = 0; f < NF; ++f) t[f] = k2 == 0 ? v[f] : t[f] + v[f];
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int j = f / (MT * 4), mm = (f / 4) % MT, q = f % 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][mm][4 * q + e] = t[f][e];
    }
    if (tid == 0) {
      if (sys) __hip_atomic_store(&cnt[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
      else __hip_atomic_store(&cnt[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }

  // epilogue: acc[j][mm][e] = C[n = n0 + 32 j + 8 (e/4) + 4 g + e%4][m = m0 + 32 mm + l32].
  // Each wavefront stages its 32 NT (n) x 64 (m) output blocks through an LDS
  // region of its own (the operand stages are free after the last barrier) as
  // fp16 rows of 32 NT outputs (CR = 4 NT 16-byte chunks), chunk c of row r at
  // position c ^ (r % CR), and then stores whole rows: lane l writes chunk
  // l % CR of row l / CR of each group of 64 / CR rows.
  uint8_t* stage = w == 0 ? (uint8_t*)&X0[0][0] : w == 1 ? (uint8_t*)&X1[0][0]
                 : w == 2 ? (uint8_t*)&W0[0][0] : (uint8_t*)&W1[0][0];
  constexpr int PASSES = MT / 2;  // 64 tokens per pass
  if constexpr (EPI != kEpiPlain) {
    auto passes = [&](auto form) {
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps)
        epi_block<EPI, NT, decltype(form)::value>(
            stage, [&](int j, int t, int e) { return acc[j][2 * ps + t][e]; }, av[ps], lane, m0 + 64 * ps, n0, M, N,
            bias, aux, act, y);
    };
    if (erf) passes(std::true_type{});
    else passes(std::false_type{});
  } else {
    constexpr int CR = 4 * NT, RB = 16 * CR;
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int nl = 32 * j + 8 * q + 4 * g;  // local output channel of e = 4 q
          float b4[4] = {0.f, 0.f, 0.f, 0.f};
          if (bias && n0 + nl < N) {
            const uint2 braw = *(const uint2*)(bias + n0 + nl);
            b4[0] = half_lo(braw.x);
            b4[1] = half_hi(braw.x);
            b4[2] = half_lo(braw.y);
            b4[3] = half_hi(braw.y);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int mm = 2 * ps + t;
            const int rl = 32 * t + l32;  // row of the staged block
            uint2 pk;
            pk.x = half_bits(acc[j][mm][4 * q + 0] + b4[0]) | (half_bits(acc[j][mm][4 * q + 1] + b4[1]) << 16);
            pk.y = half_bits(acc[j][mm][4 * q + 2] + b4[2]) | (half_bits(acc[j][mm][4 * q + 3] + b4[3]) << 16);
            const int c = nl >> 3;  // 16-byte chunk, 8-byte half (nl >> 2) & 1
            *(uint2*)(stage + rl * RB + ((c ^ (rl % CR)) << 4) + (((nl >> 2) & 1) << 3)) = pk;
          }
        }
      }
      // (the region is this wavefront's own: its LDS accesses complete in order)
#pragma unroll
      for (int rr = 0; rr < CR; ++rr) {
        const int rl = (64 / CR) * rr + lane / CR, c = lane % CR;
        const u4 v = *(const u4*)(stage + rl * RB + ((c ^ (rl % CR)) << 4));
        const int m = m0 + 64 * ps + rl, n = n0 + 8 * c;
        if (m < M && n < N) *(u4*)(y + (size_t)m * N + n) = v;
      }
    }
  }
}

// --------------------------------------------------------------------------
// prefill, layers with many output tiles: 256 (m) x 256 (n) workgroup tiles
// and one wavefront per SIMD with 256 fp32 accumulators per lane. The
// wavefront tile is 64 (n) x 256 (m) (WN = 2): each dequantized weight
// fragment feeds eight MFMAs, half the vector work per MFMA of the 64 x 128
// wavefront tiles above (measured on the MLP layer: 868 against 911 us for
// 128 x 128 wavefront tiles, WN = 4). The wavefront's own instruction stream
// overlaps the next step's dequantization with the current MFMAs. Staging,
// swizzles, the k order and the dequantization are those of w4_gemm_kernel;
// the X' stage holds 256 rows (32 KB).
// --------------------------------------------------------------------------
constexpr int GW_M = 256;
constexpr int GW_XSTAGE = GW_M * GB_K;  // halfs per X' stage (32 KB)
// groups per row up to which the wide kernel keeps all scales and zeros of its
// tile in LDS (48 KB at 64; a multiple of 16 groups, scales and zeros 16-byte
// aligned)
constexpr int kPanelGroups = 64;
// stream-K workgroups per XCD at most (one workgroup per CU: 256 CUs in 8
// XCDs)
constexpr int kSkSlots = 32;
// wide-kernel modes
constexpr int kModeTile = 0, kModeSkOne = 1, kModeSkMany = 2;

// Instruction order inside a scheduling region of 16 MFMAs: the region's ND
// LDS reads first, the first NW MFMAs alone (while those reads return), then
// each MFMA followed by up to NV vector instructions (the next step's
// dequantization); NG global loads (part of a k-tile's DMA) are spread evenly
// among the MFMAs, so that issuing the loads, which holds the wavefront's
// in-order issue, overlaps running MFMAs.
// One chunk of NM = 4 MFMAs: the chunk's ND LDS reads first, then each MFMA
// followed by up to NV vector instructions and, for the first NG, one global
// load with the scalar write of its LDS address (M0) before it.
template <int ND, int NV, int NG, int NM = 4>
__device__ __forceinline__ void sched_chunk() {
  if constexpr (ND > 0) __builtin_amdgcn_sched_group_barrier(0x100, ND, 0);
#pragma unroll
  for (int k = 0; k < NM; ++k) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (NV > 0) __builtin_amdgcn_sched_group_barrier(0x002, NV, 0);
    if (k < NG) {
      __builtin_amdgcn_sched_group_barrier(0x004, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  }
}

template <int ND, int NW, int NV, int NG, int NM = 16>
__device__ __forceinline__ void sched_order() {
  __builtin_amdgcn_sched_group_barrier(0x100, ND, 0);
#pragma unroll
  for (int k = 0; k < NM; ++k) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (k >= NW) __builtin_amdgcn_sched_group_barrier(0x002, NV, 0);
    if (NG > 0 && k % (NM / (NG > 0 ? NG : 1)) == 0) {
      __builtin_amdgcn_sched_group_barrier(0x004, 1, 0);  // the load's M0 write
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  }
}

// WN: 32-channel n tiles per wavefront (4: 128 (n) x 128 (m) wavefront tiles,
// 2: 64 (n) x 256 (m)); MTW = 16 / WN m tiles of 32 tokens.
// MODE: kModeTile, one tile per workgroup; kModeSkOne and kModeSkMany,
// stream-K (separate instantiations, so that the reduction's and the segment
// loop's registers do not weigh on the others). Stream-K: the grid is `slots` (<= kSkSlots) workgroups
// per XCD. The tiles of XCD x (its n-blocks x, x + 8, ... in the
// data-parallel order) are laid end to end as one sequence of k-tiles, and
// workgroup j of the XCD takes the j-th of `slots` equal ranges of it (even
// lengths): whole tiles,
// plus at most one partial tile at each end. The pieces of a partial tile
// meet through fp32 partial tiles in the workspace; the last to arrive adds
// them in k order and runs the epilogue.
// EPI as for w4_gemm_kernel. ROWS: the tokens, or (kModeTile) the experts' rows: an
// m-block then is a block of one expert's rows, by that expert's weights.
template <int WN, bool PANEL, int MODE, int EPI, class ROWS = AllRows>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1)))
void w4_gemm_wide_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ qw,
                         const uint16_t* __restrict__ sc, const uint8_t* __restrict__ zr,
                         const uint16_t* __restrict__ bias, uint16_t* y, int M, int N,
                         int d, int gsh, int mblk, int nblk, int slots, float* __restrict__ part,
                         uint32_t* __restrict__ cnt, int sys, const uint16_t* aux, ActForm act, int erf,
                         ROWS rows_of) {
  constexpr bool GT = epi_gated(EPI);
  static_assert(!ROWS::kExperts || MODE == kModeTile, "an expert's tile is one workgroup's");
  __shared__ __attribute__((aligned(1024))) _Float16 X0[GW_XSTAGE], X1[GW_XSTAGE], X2[GW_XSTAGE];
  __shared__ __attribute__((aligned(1024))) u4 W0[GB_WSTAGE], W1[GB_WSTAGE];
  __shared__ __attribute__((aligned(16))) uint32_t S0[GB_N], S1[GB_N], Z0[GB_N], Z1[GB_N];
  // PANEL: the tile's scales and zeros of the groups a segment's k-tiles span
  // (from the 8-aligned group below its first), loaded once per segment and
  // stored group-major ([group][256 rows]), so that the 32 rows one read
  // spans are consecutive in LDS
  __shared__ __attribute__((aligned(1024))) uint16_t SPT[PANEL ? GB_N * kPanelGroups : 8];
  __shared__ __attribute__((aligned(1024))) uint8_t ZPT[PANEL ? GB_N * kPanelGroups : 16];
  constexpr bool SK = MODE != kModeTile;
  const int tid_k = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(tid_k >> 6);  // wavefront 0..3
  constexpr int NWAV = 8 / WN;                              // wavefronts along n
  const int wn = w % NWAV, wm = w / NWAV;                   // the wavefront's n and m blocks
  // XCD-aware tile order, as in w4_gemm_kernel
  const int xcd = blockIdx.x & 7;
  const int nbx = ROWS::kExperts ? 1 : (nblk - xcd + 7) >> 3;  // (experts: find_tile_halves says where)
  if (nbx <= 0) return;
  const int groups = d >> (6 + gsh);
  const int L = d / GB_K;  // k-tiles per tile
  const uint32_t one = fp16_1024_pair();
  // SK: range j of this XCD's sequence of k-tiles starts at rstart(j)
  // (`slots` ranges of H / slots k-tile pairs, rounded down); owner(u) is
  // the range holding k-tile u (the host keeps every range non-empty)
  const int jw = blockIdx.x >> 3;
  const int64_t H = SK ? (int64_t)nbx * mblk * L / 2 : 1;
  auto rstart = [&](int j) -> int64_t { return 2 * (((int64_t)j * H) / slots); };
  auto owner = [&](int64_t u) -> int {
    int j = (int)min((int64_t)slots - 1, (u / 2) * slots / H);
    while (j + 1 < slots && rstart(j + 1) <= u) ++j;
    while (j > 0 && rstart(j) > u) --j;
    return j;
  };

  // One segment: k-tiles kt0 .. kt0 + KT - 1 (KT even) of the tile at row m0 and
  // n-block nb, the XCD's tile tl; first: the workgroup's first segment. The tile
  // has 256 rows, or half as many (H2, for an expert's last rows).
  auto segment = [&](auto h2_, const int m0, const int nb, const int kt0, const int KT, const int tl, const bool first) {
  constexpr int H2 = decltype(h2_)::value ? 2 : 1;
  constexpr int MTW = 16 / WN / H2, XD = 8 / H2;  // m tiles; X' DMAs per lane and k-tile
  // the lane index through an opaque copy, so that nothing derived from it is
  // hoisted out of the segment loop and held (spilled) across the k-loop
  int tid_o = tid_k;
  asm volatile("" : "+v"(tid_o));
  const int tid = tid_o, lane = tid & 63, l32 = lane & 31, g = lane >> 5;
  const int nw0 = nb * (GT ? GB_N / 2 : GB_N);
  const int pg0 = PANEL ? ((kt0 >> gsh) & ~7) : 0;  // first group of the panel

  // buffer resources at the tile's first row (byte offsets < 2^31: d <= 2^21,
  // checked on the host); rows past M or N are clamped to the last row
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(x + (ROWS::kGather ? 0 : (size_t)m0 * d)), (short)0,
      (ROWS::kGather ? rows_tokens(rows_of) : min(M - m0, GW_M)) * d * 2, kRsrcWord3);
  const int wrows = weight_rows<GT>(N, nw0, GB_N);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(qw + (size_t)nw0 * (d >> 1)), (short)0, wrows * (d >> 1), kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(sc + (size_t)nw0 * groups), (short)0, wrows * groups * 2, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rz = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(zr + (size_t)nw0 * groups), (short)0, wrows * groups, kRsrcWord3);
  // X' DMA c (0..7) of wavefront w fills tile rows 8 (8 w + c) .. + 7
  uint32_t xoff[8];
#pragma unroll
  for (int c = 0; c < XD; ++c) {
    const int r = 8 * (XD * w + c) + (lane >> 3);
    const int row = source_row(rows_of, m0, min(r, M - 1 - m0));
    xoff[c] = (uint32_t)(row * d + 8 * ((lane & 7) ^ ((r >> 1) & 7))) * 2u;
  }
  // code DMA c (0..1) of wavefront w fills tile rows 32 (2 w + c) .. + 31
  uint32_t woff[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int r = 32 * (2 * w + c) + (lane >> 1);
    const int row = weight_row<GT>(r, N, nw0);
    woff[c] = (uint32_t)(row * (d >> 1) + 16 * ((lane & 1) ^ ((r >> 3) & 1)));
  }
  // group scale and zero: lane l of wavefront w fetches row 64 w + l
  const uint32_t szrow = (uint32_t)(weight_row<GT>(64 * w + lane, N, nw0) * groups);

  // the DMA of one k-tile: the X' rows in two halves of four load-to-LDS
  // instructions per lane, then the codes (two) and, without PANEL, the scales
  // and zeros (two more)
  auto dma_x = [&](int half, int ktl, _Float16* xs) {
#pragma unroll
    for (int c = XD / 2 * half; c < XD / 2 * (half + 1); ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)&xs[(XD * w + c) * 64 * 8], 16, xoff[c],
                                               (kt0 + ktl) * GB_K * 2, 0, 0);
  };
  auto dma_w = [&](int ktl, u4* ws, uint32_t* ss_l, uint32_t* zs_l) {
    const int kt = kt0 + ktl;  // global k-tile
#pragma unroll
    for (int c = 0; c < 2; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)&ws[(2 * w + c) * 64], 16, woff[c], kt * (GB_K / 2), 0,
                                               0);
    if constexpr (!PANEL) {
      const uint32_t gi = (uint32_t)(kt >> gsh);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)&ss_l[64 * w], 2, (szrow + gi) * 2u, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rz, (lds_void*)&zs_l[64 * w], 1, szrow + gi, 0, 0, 0);
    }
  };

  // (arrays are sized for the largest WN and MTW and used up to WN, MTW: the
  // host pass of hipcc cannot instantiate lambdas capturing arrays of
  // template-dependent size)
  f16v acc[4][8];  // [n tile j][m tile mm]
#pragma unroll
  for (int j = 0; j < WN; ++j)
#pragma unroll
    for (int mm = 0; mm < MTW; ++mm)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[j][mm][e] = 0.0f;

  // A k-tile's per-row operands: the 32 codes of each of the wavefront's WN
  // n tiles and their group's scale and zero, in the forms dequant8 takes.
  struct Params {
    u4 wf[4];
    h2 ss[4], zz[4], zz64[4];
  };
  // the LDS reads of the operands (raw scale and zero words), then their
  // conversion
  struct Raw {
    u4 wf[4];
    uint32_t s[4], z[4];
  };
  auto read_raw = [&](int ktl, const u4* wl, const uint32_t* ss_l, const uint32_t* zs_l, Raw& q) {
    const int gi = (kt0 + ktl) >> gsh;
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      const int r = 32 * WN * wn + 32 * j + l32;
      q.wf[j] = wl[2 * r + (g ^ ((r >> 3) & 1))];
      if constexpr (PANEL) {
        q.s[j] = SPT[(gi - pg0) * GB_N + r];
        q.z[j] = ZPT[(gi - pg0) * GB_N + r];
      } else {
        q.s[j] = ss_l[r];
        q.z[j] = zs_l[r];
      }
    }
  };
  auto convert = [&](const Raw& q, Params& p) {
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      p.wf[j] = q.wf[j];
      p.ss[j] = splat2(__builtin_bit_cast(_Float16, (uint16_t)(q.s[j] & 0xffffu)));
      const float zf = (float)(q.z[j] & 0xffu);
      p.zz[j] = splat2((_Float16)(1024.0f + zf));
      p.zz64[j] = splat2((_Float16)(64.0f + zf));
    }
  };
  auto load_params = [&](int kt, const u4* wl, const uint32_t* ss_l, const uint32_t* zs_l, Params& p) {
    Raw q;
    read_raw(kt, wl, ss_l, zs_l, q);
    convert(q, p);
  };
  // X' fragments of MFMA step i (0..3) of a k-tile for the MTW m tiles
  auto read_b = [&](const _Float16* xb, int i, h8* bf) {
#pragma unroll
    for (int mm = 0; mm < MTW; ++mm) {
      const int r = 32 * MTW * wm + 32 * mm + l32;
      bf[mm] = *(const h8*)(xb + r * GB_K + 8 * ((4 * g + i) ^ ((r >> 1) & 7)));
    }
  };
  auto deq = [&](const Params& p, int i, h8* af) {
#pragma unroll
    for (int j = 0; j < WN; ++j) af[j] = dequant8(p.wf[j][i], p.zz[j], p.zz64[j], p.ss[j], one);
  };
  auto mma = [&](const h8* af, const h8* bf) {
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int mm = 0; mm < MTW; ++mm)
        acc[j][mm] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[j], bf[mm], acc[j][mm], 0, 0, 0);
  };
  // the q-th quarter of the MFMAs of one step (j major)
  constexpr int Q4 = WN * MTW / 4;
  auto mma4 = [&](int q, const h8* af, const h8* bf) {
#pragma unroll
    for (int f = Q4 * q; f < Q4 * (q + 1); ++f)
      acc[f / MTW][f % MTW] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[f / MTW], bf[f % MTW], acc[f / MTW][f % MTW], 0, 0, 0);
  };
  // Pipeline: while the MFMAs of step i of k-tile kt run, the wavefront reads
  // and dequantizes the operands of step i + 1. After step 2 it waits for the
  // DMA of k-tile kt + 1 and the barrier, so that step 3 overlaps the first
  // operands of kt + 1 (read from the other stage). Past that barrier every
  // wavefront has read all it needs of k-tile kt: step 3 sends the codes of kt +
  // 2 into kt's stage, and steps 0 and 1 of the next k-tile the X' rows of kt +
  // 3 into kt's X' stage, of which there are three. The loads of four
  // wavefronts pass at 64 bytes a cycle; all of them in step 3, as two X' stages
  // would have it, take longer than its MFMAs. Past the last tile the DMA
  // reloads the last tile, which is read but not used.
  Params P, Pn;
  h8 a[4], b[8], an[4], bn[8];
  // k-tile kt in (xb, wl, sb, zb), kt + 1 in (xn, wnx, sn, zn); xp: the X' stage
  // of kt - 1, which kt + 2 takes
  auto tile = [&](int kt, _Float16* xp, const _Float16* xb, u4* wl, uint32_t* sb, uint32_t* zb, const _Float16* xn,
                  const u4* wnx, const uint32_t* sn, const uint32_t* zn) {
    const int kd = min(kt + 2, KT - 1);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (i < 2) dma_x(i, kd, xp);
      read_b(xb, i + 1, bn);
      deq(P, i + 1, an);
      mma(a, b);
      if (i < 2) sched_order<MTW, 0, H2 * WN + 1, XD / 2, 4 * Q4>();
      else sched_order<MTW, 0, H2 * WN + 1, 0, 4 * Q4>();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if (t < WN) a[t] = an[t];
        if (t < MTW) b[t] = bn[t];
      }
    }
    // still on their way: the X' rows of kt + 2
    __builtin_amdgcn_s_waitcnt(H2 == 1 ? kWaitVm8Lgkm0 : kWaitVm4Lgkm0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // step 3 in four chunks of four MFMAs, the first with the codes' DMA of kt +
    // 2, each with a share of kt + 1's operand work
    Raw raw;
    read_raw(kt + 1, wnx, sn, zn, raw);
    read_b(xn, 0, bn);
    mma4(0, a, b);
    dma_w(kd, wl, sb, zb);
    sched_chunk<MTW + 3 * WN, 0, PANEL ? 2 : 4, Q4>();
    __builtin_amdgcn_sched_barrier(0);
    convert(raw, Pn);
    mma4(1, a, b);
    sched_chunk<0, H2 * 3 * WN, 0, Q4>();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < WN / 2; ++j) an[j] = dequant8(Pn.wf[j][0], Pn.zz[j], Pn.zz64[j], Pn.ss[j], one);
    mma4(2, a, b);
    sched_chunk<0, (13 * WN / 2 + Q4 - 1) / Q4, 0, Q4>();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = WN / 2; j < WN; ++j) an[j] = dequant8(Pn.wf[j][0], Pn.zz[j], Pn.zz64[j], Pn.ss[j], one);
    mma4(3, a, b);
    sched_chunk<0, (13 * WN / 2 + Q4 - 1) / Q4, 0, Q4>();
    __builtin_amdgcn_sched_barrier(0);
    P = Pn;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t < WN) a[t] = an[t];
      if (t < MTW) b[t] = bn[t];
    }
  };

  if constexpr (PANEL) {
    // lane l of wavefront w loads the scales (fp16) and zeros (bytes) of the
    // panel's pg groups of tile row 64 w + l, its own row, in 16-byte pieces
    // (the last piece may run into the next groups or row, which are stored
    // but never read; past the tile's rows it reads zero), and stores them
    // group-major
    const __amdgpu_buffer_rsrc_t rsp = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(sc + (size_t)nw0 * groups), (short)0, wrows * groups * 2, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rzp = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(zr + (size_t)nw0 * groups), (short)0, wrows * groups, kRsrcWord3);
    const int rr = 64 * w + lane;
    const int gr = (GT ? weight_row<GT>(rr, N, nw0) : rr) * groups;
    const int pg = ((kt0 + KT - 1) >> gsh) - pg0 + 1;  // at most kPanelGroups (checked on the host)
    u4 sv[kPanelGroups / 8], zv[kPanelGroups / 16];
#pragma unroll
    for (int c = 0; c < kPanelGroups / 8; ++c)
      if (c < (pg + 7) / 8)
        sv[c] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rsp, (gr + pg0) * 2 + 16 * c, 0, 0));
#pragma unroll
    for (int c = 0; c < kPanelGroups / 16; ++c)
      if (c < (pg + 15) / 16)
        zv[c] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rzp, gr + pg0 + 16 * c, 0, 0));
#pragma unroll
    for (int c = 0; c < kPanelGroups / 8; ++c)
      if (c < (pg + 7) / 8) {
#pragma unroll
        for (int t = 0; t < 8; ++t) SPT[(8 * c + t) * GB_N + rr] = (uint16_t)(sv[c][t >> 1] >> (16 * (t & 1)));
      }
#pragma unroll
    for (int c = 0; c < kPanelGroups / 16; ++c)
      if (c < (pg + 15) / 16) {
#pragma unroll
        for (int t = 0; t < 16; ++t) ZPT[(16 * c + t) * GB_N + rr] = (uint8_t)(zv[c][t >> 2] >> (8 * (t & 3)));
      }
  }
  dma_x(0, 0, X0);
  dma_x(1, 0, X0);
  dma_w(0, W0, S0, Z0);
  __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
  __builtin_amdgcn_s_barrier();
  dma_x(0, 1, X1);  // (KT is even: there is a second k-tile)
  dma_x(1, 1, X1);
  dma_w(1, W1, S1, Z1);
  load_params(0, W0, S0, Z0, P);
  read_b(X0, 0, b);
  deq(P, 0, a);
  int kt = 0;
  for (; kt + 6 <= KT; kt += 6) {  // the period of both rings; KT even (checked on the host)
    tile(kt, X2, X0, W0, S0, Z0, X1, W1, S1, Z1);
    tile(kt + 1, X0, X1, W1, S1, Z1, X2, W0, S0, Z0);
    tile(kt + 2, X1, X2, W0, S0, Z0, X0, W1, S1, Z1);
    tile(kt + 3, X2, X0, W1, S1, Z1, X1, W0, S0, Z0);
    tile(kt + 4, X0, X1, W0, S0, Z0, X2, W1, S1, Z1);
    tile(kt + 5, X1, X2, W1, S1, Z1, X0, W0, S0, Z0);
  }
  if (kt < KT) {
    tile(kt, X2, X0, W0, S0, Z0, X1, W1, S1, Z1);
    tile(kt + 1, X0, X1, W1, S1, Z1, X2, W0, S0, Z0);
  }
  if (kt + 2 < KT) {
    tile(kt + 2, X1, X2, W0, S0, Z0, X0, W1, S1, Z1);
    tile(kt + 3, X2, X0, W1, S1, Z1, X1, W0, S0, Z0);
  }
  // the last tile's step 3 read a stage that the epilogue below overwrites
  __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
  __builtin_amdgcn_s_barrier();

  if constexpr (SK) {
    if (KT != L) {
      // A partial tile: the workgroup stores its fp32 partial tile (wavefront
      // w's 256 accumulators per lane as [w][64 groups of 4][lane], 256 KB) in
      // its slot (0: its first segment, 1: its last; only those two can be
      // partial) and counts itself in on the counter of the tile's first
      // range; the last piece to arrive adds the pieces in range order (so
      // the sum does not depend on the order of arrival), resets the counter
      // and runs the epilogue. The ranges of a tile are those of one XCD, so
      // plain stores, an L2 atomic and loads that skip the per-CU cache
      // suffice; where the dispatch rule is not established (sys) they go
      // through memory.
      const size_t tile_floats = (size_t)GW_M * GB_N;
      auto rsrc = [&](int j, int slot) {
        return __builtin_amdgcn_make_buffer_rsrc(
            (void*)(part + ((size_t)(xcd * kSkSlots + j) * 2 + slot) * tile_floats), (short)0,
            (int)(tile_floats * 4), kRsrcWord3);
      };
      const __amdgpu_buffer_rsrc_t rmine = rsrc(jw, first ? 0 : 1);
#pragma unroll
      for (int f = 0; f < 64; ++f) {
        const int j = f >> 5, mm = (f >> 2) & 7, q = f & 3;
        const u4 v = __builtin_bit_cast(u4, f4{acc[j][mm][4 * q], acc[j][mm][4 * q + 1], acc[j][mm][4 * q + 2],
                                               acc[j][mm][4 * q + 3]});
        const int off = ((w * 64 + f) * 64 + lane) * 16;
        if (sys) __builtin_amdgcn_raw_buffer_store_b128(v, rmine, off, 0, kAuxSysW);
        else __builtin_amdgcn_raw_buffer_store_b128(v, rmine, off, 0, 0);
      }
      const int ja = owner((int64_t)tl * L);
      const int pieces = owner((int64_t)tl * L + L - 1) - ja + 1;
      const int ctr = xcd * slots + ja;
      __builtin_amdgcn_s_waitcnt(0);  // this wavefront's stores have reached L2 / memory
      __syncthreads();
      volatile uint32_t& s_last = *(uint32_t*)W0;  // (the stages take all of LDS, and the epilogue uses X0)
      if (tid == 0) {
        uint32_t old;
        if (sys) old = __hip_atomic_fetch_add(&cnt[ctr], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
        else old = __hip_atomic_fetch_add(&cnt[ctr], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = old == (uint32_t)(pieces - 1);
      }
      __syncthreads();
      if (!s_last) return;
      // the first piece is range ja's first segment if the tile is the first
      // of that range, else its last
      const int slot0 = rstart(ja) / L == tl ? 0 : 1;
      // 16 groups of 4 accumulators at a time, summed in range order from the
      // stored partial tiles (this workgroup's own included)
#pragma unroll
      for (int f0 = 0; f0 < 64; f0 += 16) {
        f4 r[16];
        for (int p = 0; p < pieces; ++p) {
          const __amdgpu_buffer_rsrc_t rk = rsrc(ja + p, p == 0 ? slot0 : 0);
          f4 v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int off = ((w * 64 + f0 + e) * 64 + lane) * 16;
            v[e] = __builtin_bit_cast(f4, sys ? __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, kAuxSysW)
                                              : __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, kAuxL2R));
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) r[e] = p == 0 ? v[e] : r[e] + v[e];
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int f = f0 + e, j = f >> 5, mm = (f >> 2) & 7, q = f & 3;
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[j][mm][4 * q + c] = r[e][c];
        }
      }
      if (tid == 0) {
        if (sys) __hip_atomic_store(&cnt[ctr], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
        else __hip_atomic_store(&cnt[ctr], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }

  // epilogue: acc[j][mm][e] = C[n = n0 + 32 j + 8 (e/4) + 4 g + e%4][m = mw0 + 32 mm + l32],
  // staged per wavefront through an 8 KB LDS region of its own (a quarter of
  // the X' stage 0, free after the last barrier) in 64 x 64 blocks, as in
  // w4_gemm_kernel
  const int n0 = nw0 + (GT ? 16 : 32) * WN * wn, mw0 = m0 + 32 * MTW * wm;
  uint8_t* stage = (uint8_t*)X0 + 8192 * w;
  if constexpr (EPI == kEpiShare) {
    float share[8];
#pragma unroll
    for (int mm = 0; mm < MTW; ++mm) share[mm] = rows_of.weight(min(mw0 + 32 * mm + l32, M - 1));
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + 32 * j + 8 * q + 4 * g;
        if (n < N) {
#pragma unroll
          for (int mm = 0; mm < MTW; ++mm) {
            const int m = mw0 + 32 * mm + l32;
            if (m < M)
              epi_share(f4{acc[j][mm][4 * q], acc[j][mm][4 * q + 1], acc[j][mm][4 * q + 2], acc[j][mm][4 * q + 3]},
                        share[mm], m, n, N, bias, (float*)y);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  } else if constexpr (EPI != kEpiPlain) {
    // blocks of 64 tokens by two tiles, the second operand two blocks ahead
    constexpr int PS = MTW / 2, BLOCKS = WN / 2 * PS;
    u4 av[2][8];
    auto fetch = [&](int b) {
      epi_fetch<EPI, 2>(av[b & 1], lane, mw0 + 64 * (b % PS), n0 + (GT ? 32 : 64) * (b / PS), M, N, aux);
    };
    fetch(0);
    fetch(1);
    auto passes = [&](auto form) {
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) {
        epi_block<EPI, 2, decltype(form)::value>(
            stage, [&](int j, int t, int e) { return acc[2 * (b / PS) + j][2 * (b % PS) + t][e]; }, av[b & 1], lane,
            mw0 + 64 * (b % PS), n0 + (GT ? 32 : 64) * (b / PS), M, N, bias, aux, act, y);
        if (b + 2 < BLOCKS) fetch(b + 2);
      }
    };
    if (erf) passes(std::true_type{});
    else passes(std::false_type{});
  } else {
#pragma unroll
  for (int jh = 0; jh < WN / 2; ++jh) {
#pragma unroll
    for (int ps = 0; ps < MTW / 2; ++ps) {
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const int j = 2 * jh + jj;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int nl = 32 * jj + 8 * q + 4 * g;  // channel of e = 4 q inside the 64-channel block
          const int n = n0 + 64 * jh + nl;
          float b4[4] = {0.f, 0.f, 0.f, 0.f};
          if (bias && n < N) {
            const uint2 braw = *(const uint2*)(bias + n);
            b4[0] = half_lo(braw.x);
            b4[1] = half_hi(braw.x);
            b4[2] = half_lo(braw.y);
            b4[3] = half_hi(braw.y);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int mm = 2 * ps + t;
            const int rl = 32 * t + l32;
            uint2 pk;
            pk.x = half_bits(acc[j][mm][4 * q + 0] + b4[0]) | (half_bits(acc[j][mm][4 * q + 1] + b4[1]) << 16);
            pk.y = half_bits(acc[j][mm][4 * q + 2] + b4[2]) | (half_bits(acc[j][mm][4 * q + 3] + b4[3]) << 16);
            const int c = nl >> 3;
            *(uint2*)(stage + rl * 128 + ((c ^ (rl & 7)) << 4) + (((nl >> 2) & 1) << 3)) = pk;
          }
        }
      }
#pragma unroll
      for (int rr = 0; rr < 8; ++rr) {
        const int rl = 8 * rr + (lane >> 3), c = lane & 7;
        const u4 v = *(const u4*)(stage + rl * 128 + ((c ^ (rl & 7)) << 4));
        const int m = mw0 + 64 * ps + rl, n = n0 + 64 * jh + 8 * c;
        if (m < M && n < N) *(u4*)(y + (size_t)m * N + n) = v;
      }
    }
  }
  }
  };

  if constexpr (!SK) {
    // one tile per workgroup: XCD x walks all of its n-blocks for each
    // m-block in turn, so that the tiles resident on it at once span few
    // m-blocks. An X' block (256 rows) is four times the bytes of a weight
    // block, so sharing X' blocks saves more L2 misses than sharing weight
    // blocks (MLP 8192 x 4096 -> 14336: 0.792 -> 0.783 ms against super-blocks
    // of 8 m-blocks, fewer misses at the same work)
    const int idx = blockIdx.x >> 3;
    const int mb = idx / nbx;
    int nb = xcd + 8 * (idx - mb * nbx);
    if (!ROWS::kExperts && mb >= mblk) return;
    int m0 = mb * GW_M;
    if constexpr (ROWS::kExperts) {
      ExpertTile tile;
      if (!rows_of.find_tile_halves(blockIdx.x, GW_M, nblk, tile, nb)) return;
      m0 = tile.first;
      M = tile.end;
      const size_t row0 = (size_t)tile.expert * (GT ? 2 * N : N);  // the expert's first weight row
      qw += row0 * (size_t)(d >> 1);
      sc += row0 * groups;
      zr += row0 * groups;
      if (bias) bias += row0;
      // an expert's last rows, up to 128: wavefront tiles of half the height
      if (M - m0 <= GW_M / 2) {
        segment(std::true_type{}, m0, nb, 0, L, 0, true);
        return;
      }
    }
    segment(std::false_type{}, m0, nb, 0, L, 0, true);
  } else {
    // the XCD's tile t, its n-blocks walked in super-blocks of 8 m-blocks
    // (the last super-block may hold fewer)
    int64_t u = rstart(jw);
    const int64_t ue = rstart(jw + 1);
    const int tfirst = (int)(u / L);
    if constexpr (MODE == kModeSkOne) {
      // every range lies in one tile (checked on the host)
      const int t = tfirst;
      const int sb = t / (8 * nbx);
      const int rows = min(8, mblk - 8 * sb);
      const int rem = t - sb * 8 * nbx;
      segment(std::false_type{}, GW_M * (8 * sb + rem % rows), xcd + 8 * (rem / rows), (int)(u - (int64_t)t * L), (int)(ue - u), t, true);
    } else {
      while (u < ue) {
        const int t = (int)(u / L);
        const int k0 = (int)(u - (int64_t)t * L);
        const int k1 = (int)min((int64_t)L, k0 + (ue - u));
        const int sb = t / (8 * nbx);
        const int rows = min(8, mblk - 8 * sb);
        const int rem = t - sb * 8 * nbx;
        segment(std::false_type{}, GW_M * (8 * sb + rem % rows), xcd + 8 * (rem / rows), k0, k1 - k0, t, t == tfirst);
        u += k1 - k0;
        if (u < ue) {
          // the epilogue's LDS reads before the next segment's DMA and panel
          // (an LDS wait and a barrier: __syncthreads would also wait for the
          // epilogue's global stores)
          __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
          __builtin_amdgcn_s_barrier();
        }
      }
    }
  }
}

template <int KS, int MT, int NT, int EPI>
void launch_gemm(unsigned blocks, hipStream_t stream, const uint16_t* x, const uint8_t* qweight,
                 const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, uint16_t* y,
                 int64_t M, int64_t N, int64_t d, int gsh, int mblk, int nblk, int mmaj, const W4Epilogue& ep) {
  hipLaunchKernelGGL((w4_gemm_kernel<KS, MT, NT, false, EPI>), dim3(blocks), dim3(256 * KS), 0, stream, x, qweight,
                     scales, zeros, bias, y, (int)M, (int)N, (int)d, gsh, mblk, nblk, 1, nullptr, nullptr, 0,
                     mmaj, ep.aux, act_form(ep.act), ep.act == PARO_ACT_GELU);
}

}  // namespace

// Smaller-tile kernel geometry, as launch_w4_gemm chooses it: 64-token tiles
// when 128-token ones would leave most SIMDs without work, 128-channel ones
// when even those leave CUs without a workgroup; k split two or four ways
// inside the workgroup; and (nsplit > 1) across workgroups when the tiles do
// not fill the CUs.
struct SmallGemm {
  int nblk256, mblk, nblk, ksin, nsplit;
  bool half, narrow;
  int64_t tiles;
};
SmallGemm small_gemm(int64_t M, int64_t N, int64_t d);
// A stream-K split's most groups per segment panel (from the 8-aligned group
// below a segment's first k-tile's: whole tiles span all of a row's groups,
// partial ones lie at the ends of the ranges), and whether every range lies
// in one tile.
void sk_shape(int64_t nblk, int64_t mblkw, int64_t L, int gsh, int slots, int64_t* panel_groups, bool* one_tile);

// N: output channels (rows of the weight block, half of them for the gated
// epilogues); y: fp16 [M][N], [M][2 N] for kEpiGatedGrad.
template <int EPI>
hipError_t launch_w4_gemm_epi(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                              const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M,
                              int64_t N, int64_t d, int group, uint32_t* cnt, float* part, const W4Epilogue& ep,
                              hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const int64_t P = epi_gated(EPI) ? 2 * N : N;  // rows of the weight block
  const int gsh = group == 64 ? 0 : group == 128 ? 1 : 2;
  const SmallGemm sg = small_gemm(M, P, d);
  const int nblk256 = sg.nblk256, mblk = sg.mblk, nblk = sg.nblk;
  const bool half = sg.half, narrow = sg.narrow;
  // 8 XCDs, each owning every 8th n-block, walked in super-blocks of 8 m-blocks
  const int64_t nbp = (nblk + 7) / 8;
  const int64_t blocks = 8 * nbp * (((int64_t)mblk + 7) / 8) * 8;
  const bool ks2 = sg.ksin == 2, ks4 = sg.ksin == 4;
  // The smaller-tile kernel's XCD order. By n-blocks, every XCD reads all of
  // X' (2 M d bytes) and an eighth of the weights; by m-blocks, an eighth of
  // X' and all of the weights (N d / 2 bytes), which is less when N < 4 M.
  // Where X' is at least 8 MiB (twice an XCD's L2) the saved re-reads show:
  // plain GEMM, 2048 x 4096 -> 1024 35.5 -> 32.0 us, 1024 x 4096 -> 1024
  // 26.3 -> 24.8, 4096 x 4096 -> 1024 102 -> 56; 2048 x 4096 -> 4096 the same
  // (76.5 us); with X' in L2 (2048 x 1024 -> 1024, 4 MiB) by n-blocks stays
  // faster (14.1 against 16.1 us). At least 8 m-blocks, so that every XCD
  // gets one.
  const int mmaj = mblk >= 8 && P < 4 * M && 2 * M * d >= (int64_t(8) << 20);
  const unsigned g = mmaj ? 8u * (unsigned)((mblk + 7) / 8) * (unsigned)nblk : (unsigned)blocks;
  // layers with many 256 x 256 tiles take the one-wavefront-per-SIMD kernel,
  // one tile per workgroup when the tiles fill whole rounds of one workgroup
  // per CU, else stream-K when the workspace holds the partial tiles
  const GemmPlan plan = plan_w4_gemm(M, P, d);
  if (plan.wide && (!plan.sk || (cnt && part))) {
    const int mblkw = (int)((M + GW_M - 1) / GW_M);
    const int64_t L = d / GB_K;
    const int64_t groups = d >> (6 + gsh);
    const int sys = plan.sk && !xcd_dispatch_is_round_robin();
    // the scale and zero panel: at most kPanelGroups groups per segment;
    // rows of a multiple of 8 groups, scales 16-byte and zeros 8-byte aligned
    int64_t pgs = groups;
    bool one_tile = false;
    if (plan.sk) sk_shape(nblk256, mblkw, L, gsh, plan.sk_slots, &pgs, &one_tile);
    const bool panel = pgs <= kPanelGroups && groups % 8 == 0 && ((uintptr_t)scales & 15) == 0 &&
                       ((uintptr_t)zeros & 7) == 0;
    const int64_t bw = plan.sk ? 8 * plan.sk_slots : 8 * ((nblk256 + 7) / 8) * (int64_t)mblkw;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)bw), dim3(256), 0, stream, x, qweight, scales, zeros, bias, y,
                         (int)M, (int)N, (int)d, gsh, mblkw, nblk256, plan.sk_slots, part, cnt, sys, ep.aux, act_form(ep.act),
                         ep.act == PARO_ACT_GELU, AllRows{});
    };
    if (plan.sk && one_tile) {
      if (panel) go(w4_gemm_wide_kernel<kWideWN, true, kModeSkOne, EPI>);
      else go(w4_gemm_wide_kernel<kWideWN, false, kModeSkOne, EPI>);
    } else if (plan.sk) {
      if (panel) go(w4_gemm_wide_kernel<kWideWN, true, kModeSkMany, EPI>);
      else go(w4_gemm_wide_kernel<kWideWN, false, kModeSkMany, EPI>);
    } else {
      if (panel) go(w4_gemm_wide_kernel<kWideWN, true, kModeTile, EPI>);
      else go(w4_gemm_wide_kernel<kWideWN, false, kModeTile, EPI>);
    }
    return hipGetLastError();
  }
  // (with an epilogue, tiles few enough to be split go to w4_tiles_kernel)
  if constexpr (EPI == kEpiPlain) {
    if (ks4 && sg.nsplit > 1 && cnt && part) {
      const int sys = !xcd_dispatch_is_round_robin();
      hipLaunchKernelGGL((w4_gemm_kernel<4, 2, 1, true, EPI>), dim3(g * (unsigned)sg.nsplit), dim3(1024), 0, stream, x,
                         qweight, scales, zeros, bias, y, (int)M, (int)N, (int)d, gsh, mblk, nblk, sg.nsplit, part,
                         cnt, sys, mmaj, ep.aux, act_form(ep.act), ep.act == PARO_ACT_GELU);
      return hipGetLastError();
    }
  }
  if (ks4) launch_gemm<4, 2, 1, EPI>(g, stream, x, qweight, scales, zeros, bias, y, M, N, d, gsh, mblk, nblk, mmaj, ep);
  else if (narrow && ks2) launch_gemm<2, 2, 1, EPI>(g, stream, x, qweight, scales, zeros, bias, y, M, N, d, gsh, mblk, nblk, mmaj, ep);
  else if (narrow) launch_gemm<1, 2, 1, EPI>(g, stream, x, qweight, scales, zeros, bias, y, M, N, d, gsh, mblk, nblk, mmaj, ep);
  else if (half && ks2) launch_gemm<2, 2, 2, EPI>(g, stream, x, qweight, scales, zeros, bias, y, M, N, d, gsh, mblk, nblk, mmaj, ep);
  else if (half) launch_gemm<1, 2, 2, EPI>(g, stream, x, qweight, scales, zeros, bias, y, M, N, d, gsh, mblk, nblk, mmaj, ep);
  else if (ks2) launch_gemm<2, 4, 2, EPI>(g, stream, x, qweight, scales, zeros, bias, y, M, N, d, gsh, mblk, nblk, mmaj, ep);
  else launch_gemm<1, 4, 2, EPI>(g, stream, x, qweight, scales, zeros, bias, y, M, N, d, gsh, mblk, nblk, mmaj, ep);
  return hipGetLastError();
}

// The experts' product in 256 x 256 tiles, one per workgroup; y by
// row (kEpiShare: fp32). d >= 256 (two k-tiles at a time, four at least).
template <int EPI, bool GATHER>
hipError_t launch_w4_experts_wide_epi(const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                                      const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y,
                                      int64_t N, int64_t d, int group, const W4Epilogue& ep, hipStream_t stream) {
  const int64_t P = epi_gated(EPI) ? 2 * N : N;
  const int gsh = group == 64 ? 0 : group == 128 ? 1 : 2;
  const int64_t groups = d >> (6 + gsh);
  const int nblk = (int)((P + GB_N - 1) / GB_N), mblk = (int)expert_blocks(t, GW_M);
  // (an expert's scales and zeros start at a multiple of 16 rows' groups)
  const bool panel = groups <= kPanelGroups && groups % 8 == 0;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(((unsigned)nblk * (unsigned)mblk + 7) / 8 * 8 + 8), dim3(256), 0, stream, x, qweight,
                       scales, zeros, bias, (uint16_t*)y, t.R, (int)N, (int)d, gsh, mblk, nblk, 0, nullptr, nullptr, 0,
                       ep.aux, act_form(ep.act), (int)(ep.act == PARO_ACT_GELU), ExpertRows<GATHER>{t});
  };
  if (panel) go(w4_gemm_wide_kernel<kWideWN, true, kModeTile, EPI, ExpertRows<GATHER>>);
  else go(w4_gemm_wide_kernel<kWideWN, false, kModeTile, EPI, ExpertRows<GATHER>>);
  return hipGetLastError();
}

}  // namespace paro
