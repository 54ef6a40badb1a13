// gfx950 kernels for the gradient of a W4 product at its input for few tokens,
//   dx[m][k] = sum_p dz[m][p] W_hat[p][k],
// straight from the codes: with few tokens, writing W_hat^T out (w4_input_grad.hip)
// would be most of the work.
//
// The contraction runs over the weight rows p, and the matrix instructions
// want eight consecutive p of one channel in a lane. A lane therefore takes
// eight rows by eight channels, one 32-bit word of codes per row, dequantizes
// the rows and transposes the 8 x 8 block inside its own registers (32 byte
// permutations); its eight fragments, one per channel, belong to eight matrix
// products whose rows are every eighth channel. No exchange between lanes.
//
// A workgroup owns 16 TT tokens by 128 channels and one of `splits` ranges of
// p, which its wavefronts share out in chunks of 64 rows. Operands come by
// load-to-LDS DMA into the wavefront's own region:
//  * codes [64 positions][4 pieces of 32 channels], row 32 s + 8 q + i of the
//    chunk at position 32 s + 4 i + q: the 64 lanes of a read touch every bank
//    once;
//  * dz [16 TT tokens][8 pieces of 8 rows], piece p of token t at p ^ (t / 2)
//    (low three bits);
//  * the rows' scales and zeros in the forms dequant8 takes.
// The wavefronts' sums meet in LDS; those of several ranges as fp32 in the
// workspace, which a second kernel adds in range order. What bounds it: the
// latency of a chunk's loads, as few chunks follow one another (4096 rows of
// 4096, one token: 9.6 us with both launches, one chunk per wavefront); on large
// layers the stream of the codes (28672 rows of 4096: 61.5 MB in 29 us, 2.1
// TB/s), beside which the dequantization and transposition of a chunk's 8192
// codes are 360 vector instructions of a wavefront.
#include <algorithm>

#include "paro_internal.h"
#include "w4_common.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

using namespace w4;

typedef __attribute__((address_space(3))) void lds_void;
constexpr int kRsrcWord3 = 0x00020000;  // gfx9 buffer resource word 3
constexpr int kWaitVmLgkm0 = 0x70;      // s_waitcnt vmcnt(0) lgkmcnt(0)
constexpr int kCus = 256;               // compute units

constexpr int kChunk = 64;  // weight rows per chunk
constexpr int row_waves(int tt) { return tt == 1 ? 16 : 8; }
// codes, scales and zeros (two groups a row), dz; and room for a token block's sums
constexpr int row_bytes(int tt) { return std::max(8192, 4096 + 1024 + 2048 * tt); }

template <int TT>
__global__ __launch_bounds__(64 * row_waves(TT))
void w4_grad_rows_kernel(const uint8_t* __restrict__ qw, const uint16_t* __restrict__ sc,
                         const uint8_t* __restrict__ zr, const uint16_t* __restrict__ dz, int M, int P, int d,
                         int gsh, int mblk, int kblk, int splits, uint16_t* __restrict__ dx,
                         float* __restrict__ part) {
  constexpr int WB = row_bytes(TT);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[row_waves(TT) * WB];
  const int lane = threadIdx.x & 63, r = lane & 15, kq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), nw = blockDim.x >> 6;
  // token blocks fastest: they share the weights
  const int blk = blockIdx.x;
  const int mb = blk % mblk, kb = blk / mblk % kblk, sp = blk / (mblk * kblk);
  const int m0 = 16 * TT * mb, k0 = 128 * kb;
  const int chunks = (P + kChunk - 1) / kChunk;
  const int c0 = (int)((int64_t)chunks * sp / splits), c1 = (int)((int64_t)chunks * (sp + 1) / splits);
  const int sgr = d >> (6 + gsh), gi = k0 >> (6 + gsh);
  uint8_t* cl = lds + w * WB;
  uint2* tab = (uint2*)(cl + 4096);  // [64 rows][2 groups]
  uint8_t* zl = cl + 5120;
  const int tokens = min(16 * TT, M - m0);
  const __amdgpu_buffer_rsrc_t rd = __builtin_amdgcn_make_buffer_rsrc((void*)(dz + (size_t)m0 * P), (short)0,
                                                                      tokens * P * 2, kRsrcWord3);
  uint32_t doff[8];  // (tokens past M repeat the last one and are never stored)
#pragma unroll
  for (int t = 0; t < 2 * TT; ++t) {
    const int row = 8 * t + (lane >> 3);
    doff[t] = (uint32_t)(min(row, tokens - 1) * P * 2);
  }
  const int dpiece = lane & 7;
  const uint32_t one = fp16_1024_pair();
  f4 acc[8][4];
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[e][t] = f4{0.f, 0.f, 0.f, 0.f};

  for (int c = c0 + w; c < c1; c += nw) {
    const int p0 = kChunk * c, left = P - p0;  // rows of the chunk (P % 16 == 0)
    const int prow = p0 + min(lane, left - 1);
    uint32_t s0 = sc[(size_t)prow * sgr + gi], z0 = zr[(size_t)prow * sgr + gi], s1 = 0, z1 = 0;
    if (gsh == 0) {
      s1 = sc[(size_t)prow * sgr + gi + 1];
      z1 = zr[(size_t)prow * sgr + gi + 1];
    }
    const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(qw + (size_t)p0 * (d >> 1)), (short)0, min(kChunk, left) * (d >> 1), kRsrcWord3);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int q = 16 * t + (lane >> 2);
      const int row = min(32 * (q >> 5) + 8 * (q & 3) + ((q >> 2) & 7), left - 1);
      const uint32_t off = (uint32_t)(row * (d >> 1) + (k0 >> 1) + 16 * (lane & 3));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_void*)(cl + 1024 * t), 16, off, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < 2 * TT; ++t) {
      const int row = 8 * t + (lane >> 3);
      const int piece = min(dpiece ^ ((row >> 1) & 7), (left >> 3) - 1);
      const uint32_t off = doff[t] + (uint32_t)(2 * p0 + 16 * piece);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (lds_void*)(zl + 1024 * t), 16, off, 0, 0, 0);
    }
    // scale | 0, 1024 + z | 64 + z (rows past P: scale zero)
    auto form = [&](uint32_t s, uint32_t z) {
      const _Float16 ss = __builtin_bit_cast(_Float16, (uint16_t)(lane < left ? s : 0u));
      const float zf = (float)z;
      const h2 a = {ss, (_Float16)0.0f};
      const h2 b = {(_Float16)(1024.0f + zf), (_Float16)(64.0f + zf)};
      return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    };
    tab[2 * lane] = form(s0, z0);
    if (gsh == 0) tab[2 * lane + 1] = form(s1, z1);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u4 v[8];  // row 32 s + 8 kq + i, channels k0 + 8 r .. + 7
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t code = *(const uint32_t*)(cl + 64 * (32 * s + 4 * i + kq) + 4 * r);
        const uint2 q = tab[2 * (32 * s + 8 * kq + i) + (gsh == 0 ? r >> 3 : 0)];
        const h2 a = __builtin_bit_cast(h2, q.x), b = __builtin_bit_cast(h2, q.y);
        v[i] = __builtin_bit_cast(u4, dequant8(code, splat2(b[0]), splat2(b[1]), splat2(a[0]), one));
      }
      h8 bf[4];
      const bool in = 32 * s + 8 * kq < left;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        u4 raw = *(const u4*)(zl + 2048 * t + 128 * r + 16 * ((4 * s + kq) ^ ((r >> 1) & 7)));
        if (!in) raw = u4{0u, 0u, 0u, 0u};
        bf[t] = __builtin_bit_cast(h8, raw);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a[j] = __builtin_amdgcn_perm(v[2 * j + 1][e >> 1], v[2 * j][e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
        const h8 af = __builtin_bit_cast(h8, a);
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[e][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, bf[t], acc[e][t], 0, 0, 0);
      }
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kWaitVmLgkm0);  // its LDS reads, before the next chunk's DMA
    asm volatile("" ::: "memory");
  }

  // acc[e][t][j] = dx[token m0 + 16 t + r][channel k0 + 8 (4 kq + j) + e]; the
  // wavefronts' sums of a token block in wavefront order, four channels at a time
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    if (t > 0) __syncthreads();
#pragma unroll
    for (int jh = 0; jh < 8; ++jh) {
      const int j = jh >> 1, e = 4 * (jh & 1);
      *(f4*)(cl + 1024 * jh + 16 * lane) = f4{acc[e][t][j], acc[e + 1][t][j], acc[e + 2][t][j], acc[e + 3][t][j]};
    }
    __syncthreads();
    for (int jh = w; jh < 8; jh += nw) {
      const uint8_t* p = lds + 1024 * jh + 16 * lane;
      f4 sum = *(const f4*)p;
      for (int k = 1; k < nw; ++k) sum += *(const f4*)(p + k * WB);
      const int m = m0 + 16 * t + r, k = k0 + 8 * (4 * kq + (jh >> 1)) + 4 * (jh & 1);
      if (m < M) {
        if (splits > 1) {
          *(f4*)(part + ((size_t)sp * M + m) * d + k) = sum;
        } else {
          uint2 o;
          o.x = half_bits(sum[0]) | (half_bits(sum[1]) << 16);
          o.y = half_bits(sum[2]) | (half_bits(sum[3]) << 16);
          *(uint2*)(dx + (size_t)m * d + k) = o;
        }
      }
    }
  }
}

// dx = the partial sums [splits][n4][4], added in order
__global__ __launch_bounds__(256) void add_splits_kernel(const f4* __restrict__ part, int splits, int64_t n4,
                                                         uint2* __restrict__ dx) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  f4 v[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) v[s] = part[min(s, splits - 1) * n4 + i];
  f4 sum = v[0];
#pragma unroll
  for (int s = 1; s < 8; ++s)
    if (s < splits) sum += v[s];
  uint2 o;
  o.x = half_bits(sum[0]) | (half_bits(sum[1]) << 16);
  o.y = half_bits(sum[2]) | (half_bits(sum[3]) << 16);
  dx[i] = o;
}

int tokens_per_block(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }

// Ranges of p: as many as fit the CUs in one round, each wavefront a chunk at
// least, at most eight.
int row_splits(int64_t M, int64_t P, int64_t d) {
  const int tt = tokens_per_block(M);
  const int64_t blocks = (M + 16 * tt - 1) / (16 * tt) * (d / 128), chunks = (P + kChunk - 1) / kChunk;
  return (int)std::max<int64_t>(1, std::min<int64_t>({kCus / blocks, chunks / 8, 8}));
}

}  // namespace

// Up to 128 tokens: 14336 rows of 4096 at 1 / 64 / 128 tokens 64 / 66 / 72 us by
// w4_input_grad.hip against 19 / 27 / 39 here, 28672 rows of 4096 137 / 150 / 158
// against 29 / 41 / 66, 4096 of 4096 30 / 31 / 33 against 10 / 19 / 22; at 192
// tokens 34 against 38 (4096 of 4096), 185 against 126. Every 64 tokens dequantize
// all of the weights again.
bool input_grad_rows_fit(int64_t M) { return M <= 128; }

size_t input_grad_rows_bytes(int64_t M, int64_t P, int64_t d) {
  const int splits = row_splits(M, P, d);
  return splits > 1 ? (size_t)splits * M * d * 4 : 0;
}

hipError_t launch_w4_input_grad_rows(const uint16_t* dz, const uint8_t* qweight, const uint16_t* scales,
                                     const uint8_t* zeros, uint16_t* dx, int64_t M, int64_t P, int64_t d, int group,
                                     void* scratch, hipStream_t stream) {
  const int gsh = group == 64 ? 0 : group == 128 ? 1 : 2;
  const int tt = tokens_per_block(M), splits = row_splits(M, P, d);
  const int mblk = (int)((M + 16 * tt - 1) / (16 * tt)), kblk = (int)(d / 128);
  const int64_t most = (P + kChunk - 1) / kChunk / splits + 1;
  auto go = [&](auto kernel, int waves) {
    const int nw = (int)std::min<int64_t>(waves, most);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(mblk * kblk * splits)), dim3(64 * nw), 0, stream, qweight, scales,
                       zeros, dz, (int)M, (int)P, (int)d, gsh, mblk, kblk, splits, dx, (float*)scratch);
  };
  if (tt == 1) go(w4_grad_rows_kernel<1>, row_waves(1));
  else if (tt == 2) go(w4_grad_rows_kernel<2>, row_waves(2));
  else go(w4_grad_rows_kernel<4>, row_waves(4));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int64_t n4 = M * d / 4;
  hipLaunchKernelGGL(add_splits_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, stream, (const f4*)scratch,
                     splits, n4, (uint2*)dx);
  return hipGetLastError();
}

}  // namespace paro
