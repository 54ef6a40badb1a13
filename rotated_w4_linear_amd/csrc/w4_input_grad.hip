// gfx950 kernels for the gradient of a W4 product at its input,
//   dX'[m][k] = sum_p dZ[m][p] W_hat[p][k],
// W_hat[p][k] the fp16 number nearest to (q - z) s, P rows of weights.
// The contraction runs over the weight rows, along which neither the packed
// codes nor W_hat are contiguous, so W_hat^T [k][p] is written out first
// (dequantized and transposed through LDS, fp16, p padded with zeros to a
// multiple of 64) and the product is then a dense "NT" one (dense_gemm.hip).
// W_hat^T costs 2.5 P d bytes written and read whatever M is.
#include "paro_internal.h"
#include "w4_common.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

using namespace w4;

constexpr int TP = 128, TD = 128;  // weight rows and channels per workgroup
constexpr int TS = TP / 2 + 4;     // LDS words per channel: two rows a word, rows 16-byte aligned

// wt[k][p] (row stride pp, a multiple of 64): 128 rows x 128 channels per
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
      v[b][i] = dequant8(c[i], splat2((_Float16)(1024.0f + z)), ss, splat2((_Float16)(1024.0f + 16.0f * z)),
                         ss * splat2((_Float16)0.0625f), one);
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
    if (p0 + 8 * c < pp) *(u4*)(wt + (size_t)(k0 + kk) * pp + p0 + 8 * c) = *(const u4*)&t[kk * TS + 4 * c];
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

size_t a256(size_t b) { return (b + 255) & ~(size_t)255; }
int64_t pad64(int64_t n) { return (n + 63) & ~int64_t(63); }

}  // namespace

size_t input_grad_scratch_bytes(int64_t M, int64_t P, int64_t d) {
  const int64_t pp = pad64(P);
  return a256((size_t)d * pp * 2) + (pp != P ? a256((size_t)M * pp * 2) : 0);
}

hipError_t launch_w4_input_grad(const uint16_t* dz, const uint8_t* qweight, const uint16_t* scales,
                                const uint8_t* zeros, uint16_t* dx, int64_t M, int64_t P, int64_t d, int group,
                                void* ws, hipStream_t stream) {
  const int gsh = group == 64 ? 0 : group == 128 ? 1 : 2;
  const int64_t pp = pad64(P);
  uint16_t* wt = (uint16_t*)ws;
  const dim3 grid((unsigned)(d / TD), (unsigned)((pp + TP - 1) / TP));
  hipLaunchKernelGGL(w4_transpose_kernel, grid, dim3(256), 0, stream, qweight, scales, zeros, (int)P, (int)d, gsh, wt,
                     (int)pp);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (pp != P) {  // the product's k-tiles are 64 wide: whole ones, so that no row reads its neighbour
    uint16_t* padded = (uint16_t*)((char*)ws + a256((size_t)d * pp * 2));
    const int64_t blocks = (M * (pp / 8) + 255) / 256;
    hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, stream,
                       (const u4*)dz, M, (int)(P / 8), (u4*)padded, (int)(pp / 8));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    dz = padded;
  }
  return launch_nt_gemm_f16(dz, pp, wt, pp, M, d, pp, dx, d, stream);
}

}  // namespace paro
