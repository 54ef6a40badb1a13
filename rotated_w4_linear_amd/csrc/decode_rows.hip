// gfx950 kernel for the W4 products with an epilogue on at most 16 tokens whose
// activations are transformed already (w4_epilogue.h: act and gated).
//
// The layer is a stream over the packed weights. A workgroup owns 16 output
// channels (gated: their 16 gate and 16 up rows) over the whole of k, which its
// wavefronts share out in chunks of 512: every sum stays inside the workgroup
// and is added up in LDS, with no partial sums in memory and no counters. (The
// kernel of w4_decode_kernels.h, which transforms as well and therefore wants
// many rows per transformed segment, splits k over workgroups: 14336 -> 4096 at
// 16 tokens then moves 7 MB of partial sums, which 32 workgroups add up at the
// end.) With 16 rows per workgroup each CU reads all of X', 16 tokens at most,
// from L2.
//
// Operands go from global memory straight into LDS (16-byte load-to-LDS DMA),
// into a region of the wavefront's own, so no barrier is needed before they are
// read. That is for the access pattern: a v_mfma_f32_16x16x32_f16 operand has a
// different row in each of 16 neighbouring lanes, and loading it straight into
// registers looks up 64 cache lines for 1 KB; a DMA instruction takes 4 weight
// rows of 256 bytes, or 1 KB of one token. (Loads into registers: 21.5 us for
// 14336 -> 4096 at 16 tokens.)
//  * codes [16 rows][16 pieces of 32 codes], piece p of row r at p ^ r;
//  * X' [MT tokens][64 pieces of 8 channels], piece p of token t at p ^ t (low
//    four bits): 16 lanes of an operand read hit 16 positions modulo 16.
// MT: tokens staged (1, 4 or 16); operand columns past it repeat token r % MT,
// and columns past M are not stored.
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

// LDS bytes of a wavefront, and wavefronts per workgroup at most: two
// workgroups fit a CU up to 4 tokens, one with 16
constexpr int wave_bytes(bool gated, int mt) { return (gated ? 8192 : 4096) + 1024 * mt; }
constexpr int max_waves(bool gated, int mt) { return mt == 1 ? (gated ? 8 : 16) : mt == 4 ? (gated ? 6 : 10) : (gated ? 6 : 7); }

// SZV: group 128 and whole chunks, so that a row's four scales and four zeros
// of a chunk are one 8-byte and one 4-byte load.
template <int EPI, int MT, bool SZV>
__global__ __launch_bounds__(64 * max_waves(epi_gated(EPI), MT))
void w4_rows_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ qw,
                    const uint16_t* __restrict__ sc, const uint8_t* __restrict__ zr,
                    const uint16_t* __restrict__ bias, uint16_t* y, int M, int N, int d, int gsh, int nblk, int per,
                    const uint16_t* aux, ActForm act, int erf) {
  constexpr bool GT = epi_gated(EPI);
  constexpr int TJ = GT ? 2 : 1, WB = wave_bytes(GT, MT), NW = max_waves(GT, MT);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NW * WB];
  // neighbouring channels on one XCD: they share output lines
  const int blk = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (blk >= nblk) return;
  const int lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), nw = blockDim.x >> 6;
  uint8_t* wl = lds + w * WB;
  uint8_t* xl = wl + 4096 * TJ;
  const int c0 = 16 * blk;
  const int segs = d >> 7, chunks = (segs + 3) >> 2;
  const int sgr = d >> (6 + gsh);  // quantization groups per row
  const bool token = r < M;
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc((void*)x, (short)0, M * d * 2, kRsrcWord3);
  auto rows = [&](int j) {  // the block's rows of tile j (rows past N repeat the last one and are never stored)
    return __builtin_amdgcn_make_buffer_rsrc((void*)(qw + ((size_t)c0 + (size_t)j * N) * (size_t)(d >> 1)), (short)0,
                                             min(16, N - c0) * (d >> 1), kRsrcWord3);
  };
  const uint32_t one = fp16_1024_pair();
  f4 acc[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) acc[j] = f4{0.f, 0.f, 0.f, 0.f};

  for (int c = w; c < chunks; c += nw) {
    const int nq = SZV ? 4 : min(4, segs - 4 * c);  // groups of 128 in the chunk
    // scales and zeros of row r, one load per row (kq = 0)
    uint2 s4[TJ];
    uint32_t z4[TJ], sraw[TJ][4], zraw[TJ][4];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const size_t grow = ((size_t)min(c0 + r, N - 1) + (size_t)j * N) * sgr;
      if constexpr (SZV) {
        s4[j] = make_uint2(0u, 0u);
        z4[j] = 0u;
        if (kq == 0) {
          s4[j] = *(const uint2*)(sc + grow + 4 * c);
          z4[j] = *(const uint32_t*)(zr + grow + 4 * c);
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          // this lane's 32 codes share one group (groups past the end of d: never used)
          const int gi = (128 * min(4 * c + g, segs - 1) + 32 * kq) >> (6 + gsh);
          sraw[j][g] = sc[grow + gi];
          zraw[j][g] = zr[grow + gi];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const __amdgpu_buffer_rsrc_t rw = rows(j);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int row = 4 * b + kq, piece = min((lane & 15) ^ row, 4 * nq - 1);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(wl + 4096 * j + 1024 * b), 16,
                                                 min(row, N - 1 - c0) * (d >> 1) + 16 * piece, 256 * c, 0, 0);
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int piece = min((lane & 48) | ((lane ^ t) & 15), 16 * nq - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(xl + 1024 * t), 16, min(t, M - 1) * d * 2 + 16 * piece,
                                               1024 * c, 0, 0);
    }
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
    if constexpr (SZV) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const uint32_t lo = __shfl((int)s4[j].x, r), hi = __shfl((int)s4[j].y, r), zz = __shfl((int)z4[j], r);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          sraw[j][g] = ((g < 2 ? lo : hi) >> (16 * (g & 1))) & 0xffffu;
          zraw[j][g] = (zz >> (8 * g)) & 0xffu;
        }
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (SZV || g < nq) {
        h8 b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = r % MT, p = 16 * g + 4 * kq + i;
          b[i] = *(const h8*)(xl + 1024 * t + 16 * ((p & 48) | ((p ^ t) & 15)));
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          const u4 v = *(const u4*)(wl + 4096 * j + 256 * r + 16 * ((4 * g + kq) ^ r));
          const h2 ss = splat2(__builtin_bit_cast(_Float16, (uint16_t)sraw[j][g]));
          const float zf = (float)zraw[j][g];
          const h2 zz = splat2((_Float16)(1024.0f + zf)), zz64 = splat2((_Float16)(64.0f + zf));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(dequant8(v[i], zz, zz64, ss, one), b[i], acc[j], 0, 0, 0);
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);  // its LDS reads, before the next chunk's DMA
  }

  // the wavefronts' sums, added in wavefront order by the first one:
  // acc[j][e] = Z[m = r][channel c0 + 4 kq + e] (j: gate, up)
  // (each leaves them in its own region)
#pragma unroll
  for (int j = 0; j < TJ; ++j) *(f4*)(wl + 1024 * j + 16 * lane) = acc[j];
  __syncthreads();
  if (w != 0) return;
  f4 z[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) z[j] = acc[j];
  for (int k = 1; k < nw; ++k)
#pragma unroll
    for (int j = 0; j < TJ; ++j) z[j] += *(const f4*)(lds + k * WB + 1024 * j + 16 * lane);
  if (token && c0 + 4 * kq < N) epi_lane<EPI>(z, r, c0 + 4 * kq, N, bias, aux, act, erf, y);
}

// The same for layers with more 16-channel blocks than CUs: one workgroup per
// CU goes from block to block. Its wavefronts keep their R chunks of k for
// good, the X' operands of those in registers, and a wavefront's next codes
// come into the other of its two LDS buffers while it multiplies. A workgroup
// per block would read X' once per block: 4096 -> 14336 at 16 tokens 23.0 us
// against 12.3, gated 30.6 against 19.1; at 1 token 11.7 and 11.1, gated 17.6
// and 18.3. The weights alone stream in 9.7 us (gated, with the launch); their
// dequantization takes 6.5 us of vector instructions, overlapped in part. One
// barrier per block: the sums of a block go to one of two places in LDS, and
// wavefront (block % wavefronts) adds them while the others go on.
constexpr int stream_waves(bool gated) { return gated ? 8 : 16; }

template <int EPI, int MT, int R, bool SZV>
__global__ __launch_bounds__(64 * stream_waves(epi_gated(EPI)))
void w4_rows_stream_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ qw,
                           const uint16_t* __restrict__ sc, const uint8_t* __restrict__ zr,
                           const uint16_t* __restrict__ bias, uint16_t* y, int M, int N, int d, int gsh, int nblk,
                           int per, const uint16_t* aux, ActForm act, int erf) {
  constexpr bool GT = epi_gated(EPI);
  constexpr int TJ = GT ? 2 : 1, NW = stream_waves(GT), CB = 4096 * TJ;  // bytes of a chunk's codes
  __shared__ __attribute__((aligned(1024))) uint8_t W0[NW * CB], W1[NW * CB];
  __shared__ f4 red[2][NW * TJ * 64];
  const int xcd = blockIdx.x & 7, slots = gridDim.x >> 3;
  const int end = min(nblk, (xcd + 1) * per);
  const int lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), nw = blockDim.x >> 6;
  const int segs = d >> 7, chunks = (segs + 3) >> 2;
  const int sgr = d >> (6 + gsh);
  uint8_t* b0 = W0 + w * CB;
  uint8_t* b1 = W1 + w * CB;

  // X' operands of chunk w + nw * k: staged through the code buffers, MT or
  // 4 TJ tokens at a time
  h8 xf[R][4][4];
  {
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc((void*)x, (short)0, M * d * 2, kRsrcWord3);
    constexpr int STEP = MT < 4 * TJ ? MT : 4 * TJ;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = min(w + nw * k, chunks - 1);
      const int nq = SZV ? 4 : min(4, segs - 4 * c);
#pragma unroll
      for (int t0 = 0; t0 < MT; t0 += STEP) {
#pragma unroll
        for (int t = t0; t < t0 + STEP; ++t) {
          const int piece = min((lane & 48) | ((lane ^ t) & 15), 16 * nq - 1);
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(b0 + 1024 * (t - t0)), 16,
                                                   min(t, M - 1) * d * 2 + 16 * piece, 1024 * c, 0, 0);
        }
        __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
        const int t = r % MT;
        if (t >= t0 && t < t0 + STEP) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int p = 16 * g + 4 * kq + i;
              xf[k][g][i] = *(const h8*)(b0 + 1024 * (t - t0) + 16 * ((p & 48) | ((p ^ t) & 15)));
            }
        }
        __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
      }
    }
  }

  struct Group {  // scales and zeros of a chunk's rows
    uint2 s4[TJ];
    uint32_t z4[TJ], s[TJ][4], z[TJ][4];
  };
  auto load = [&](int blk, int k, uint8_t* buf, Group& q) {
    const int c0 = 16 * blk, c = min(w + nw * k, chunks - 1);
    const int nq = SZV ? 4 : min(4, segs - 4 * c);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(qw + ((size_t)c0 + (size_t)j * N) * (size_t)(d >> 1)), (short)0, min(16, N - c0) * (d >> 1),
          kRsrcWord3);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int row = 4 * b + kq, piece = min((lane & 15) ^ row, 4 * nq - 1);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(buf + 4096 * j + 1024 * b), 16,
                                                 min(row, N - 1 - c0) * (d >> 1) + 16 * piece, 256 * c, 0, 0);
      }
      const size_t grow = ((size_t)min(c0 + r, N - 1) + (size_t)j * N) * sgr;
      if constexpr (SZV) {
        if (kq == 0) {
          q.s4[j] = *(const uint2*)(sc + grow + 4 * c);
          q.z4[j] = *(const uint32_t*)(zr + grow + 4 * c);
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int gi = (128 * min(4 * c + g, segs - 1) + 32 * kq) >> (6 + gsh);
          q.s[j][g] = sc[grow + gi];
          q.z[j][g] = zr[grow + gi];
        }
      }
    }
  };

  const uint32_t one = fp16_1024_pair();
  f4 acc[TJ];
  // one chunk: its codes have landed in `buf`, the next ones go to `other`
  auto chunk = [&](int blk, int k, const uint8_t* buf, uint8_t* other, Group& q) {
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
    uint32_t s[TJ][4], z[TJ][4];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if constexpr (SZV) {
        const uint32_t lo = __shfl((int)q.s4[j].x, r), hi = __shfl((int)q.s4[j].y, r), zz = __shfl((int)q.z4[j], r);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          s[j][g] = ((g < 2 ? lo : hi) >> (16 * (g & 1))) & 0xffffu;
          z[j][g] = (zz >> (8 * g)) & 0xffu;
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          s[j][g] = q.s[j][g];
          z[j][g] = q.z[j][g];
        }
      }
    }
    const int nb = k + 1 < R ? blk : blk + slots, nk = k + 1 < R ? k + 1 : 0;
    if (nb < end) load(nb, nk, other, q);
    const int c = w + nw * k;
    if (R == 1 || c < chunks) {
      const int nq = SZV ? 4 : min(4, segs - 4 * c);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (SZV || g < nq) {
#pragma unroll
          for (int j = 0; j < TJ; ++j) {
            const u4 v = *(const u4*)(buf + 4096 * j + 256 * r + 16 * ((4 * g + kq) ^ r));
            const h2 ss = splat2(__builtin_bit_cast(_Float16, (uint16_t)s[j][g]));
            const float zf = (float)z[j][g];
            const h2 zz = splat2((_Float16)(1024.0f + zf)), zz64 = splat2((_Float16)(64.0f + zf));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(dequant8(v[i], zz, zz64, ss, one), xf[k][g][i], acc[j],
                                                              0, 0, 0);
          }
        }
      }
    }
  };
  int it = 0;
  // a block in (cur, alt): with R odd the buffers change places from block to block
  auto block = [&](int blk, uint8_t* cur, uint8_t* alt, Group& q) {
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[j] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < R; ++k) chunk(blk, k, k & 1 ? alt : cur, k & 1 ? cur : alt, q);
    f4* place = red[it & 1];
#pragma unroll
    for (int j = 0; j < TJ; ++j) place[(w * TJ + j) * 64 + lane] = acc[j];
    // (a barrier for what this wavefront stored to LDS: a fence would also wait
    // for the codes that are on their way there; the empty statements keep the
    // compiler from moving accesses across it)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (w == it % nw) {
      f4 z[TJ];
#pragma unroll
      for (int j = 0; j < TJ; ++j) z[j] = place[j * 64 + lane];
      for (int k = 1; k < nw; ++k)
#pragma unroll
        for (int j = 0; j < TJ; ++j) z[j] += place[(k * TJ + j) * 64 + lane];
      const int n = 16 * blk + 4 * kq;
      if (r < M && n < N) epi_lane<EPI>(z, r, n, N, bias, aux, act, erf, y);
    }
    ++it;
  };
  int blk = xcd * per + (blockIdx.x >> 3);
  if (blk >= end) return;
  Group q;
  load(blk, 0, b0, q);
  for (; blk < end; blk += 2 * slots) {
    block(blk, b0, b1, q);
    if (blk + slots < end) {
      if constexpr (R % 2) block(blk + slots, b1, b0, q);
      else block(blk + slots, b0, b1, q);
    }
  }
}

template <int EPI, int MT>
hipError_t launch(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                  const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
                  const W4Epilogue& ep, hipStream_t stream) {
  constexpr bool gated = epi_gated(EPI);
  const int gsh = group == 64 ? 0 : group == 128 ? 1 : 2;
  const int nblk = (int)((N + 15) / 16), per = (nblk + 7) / 8;
  const int chunks = (int)((d + 511) / 512);
  const bool szv = group == 128 && d % 512 == 0 && ((uintptr_t)scales & 7) == 0 && ((uintptr_t)zeros & 3) == 0;
  auto go = [&](auto kernel, unsigned blocks, int nw) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(64 * nw), 0, stream, x, qweight, scales, zeros, bias, y, (int)M,
                       (int)N, (int)d, gsh, nblk, per, ep.aux, act_form(ep.act), (int)(ep.act == PARO_ACT_GELU));
  };
  // as many wavefronts as give each the same number of chunks
  constexpr int most = stream_waves(gated);
  const int rounds = (chunks + most - 1) / most;
  if (nblk > kCus && rounds <= (gated ? 2 : 1)) {
    const int nw = (chunks + rounds - 1) / rounds;
    if constexpr (gated) {
      if (rounds == 2) {
        if (szv) go(w4_rows_stream_kernel<EPI, MT, 2, true>, kCus, nw);
        else go(w4_rows_stream_kernel<EPI, MT, 2, false>, kCus, nw);
        return hipGetLastError();
      }
    }
    if (szv) go(w4_rows_stream_kernel<EPI, MT, 1, true>, kCus, nw);
    else go(w4_rows_stream_kernel<EPI, MT, 1, false>, kCus, nw);
    return hipGetLastError();
  }
  constexpr int most1 = max_waves(gated, MT);
  const int rounds1 = (chunks + most1 - 1) / most1;
  const int nw = (chunks + rounds1 - 1) / rounds1;
  if (szv) go(w4_rows_kernel<EPI, MT, true>, 8u * (unsigned)per, nw);
  else go(w4_rows_kernel<EPI, MT, false>, 8u * (unsigned)per, nw);
  return hipGetLastError();
}

template <int EPI>
hipError_t launch_tokens(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                         const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
                         const W4Epilogue& ep, hipStream_t stream) {
  if (M == 1) return launch<EPI, 1>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
  if (M <= 4) return launch<EPI, 4>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
  return launch<EPI, 16>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
}

}  // namespace

hipError_t launch_w4_rows(bool gated, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                          const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d,
                          int group, const W4Epilogue& ep, hipStream_t stream) {
  return gated ? launch_tokens<kEpiGated>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream)
               : launch_tokens<kEpiAct>(x, qweight, scales, zeros, bias, y, M, N, d, group, ep, stream);
}

}  // namespace paro
