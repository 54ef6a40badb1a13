// gfx950 kernels for the gradient of the experts' products at their input,
//   U[r][k] = sum_p dz[r][p] W_hat[e][p][k],
// row r by its expert e, on experts with many rows (w4_input_grad_rows.hip takes
// few). dz by token (GATHER: dY of the combining product) or by row (dZ of the
// gated one).
//
// The contraction runs over the weight rows p, along which the codes are not
// contiguous. Writing W_hat^T out first, as w4_input_grad.hip does for one weight
// block, would move 4.5 bytes a weight for every expert and hold two; here a
// workgroup dequantizes and transposes the codes of its 256 channels on the way:
// a thread takes eight rows p by eight channels of a k-tile of 64 p (a 32-bit
// word of codes a row), dequantizes the rows two channels at a time and joins the
// rows' halves by byte permutations into the 16-byte fragment of each channel,
// which goes to LDS as a row of the matrix cores' first operand. 140 vector
// instructions a thread and k-tile, beside 64 MFMAs of a wavefront, each 8 issue
// slots long.
//
// Workgroup tiles of 256 channels by 64 TM rows, four wavefronts of 128 x 32 TM
// (4 x TM accumulator tiles of v_mfma_f32_32x32x16_f16). dz comes by load-to-LDS
// DMA, two stages; fragments into two stages as well:
//  * fragments [256][64 p]: channel 8 c + e of the tile at row 128 (c / 16) + 32
//    (e / 2) + 16 (e % 2) + c % 16, chunk q of 8 p at q ^ (row % 8) ^ (row / 8 % 2).
//    Reads and writes go over consecutive rows; 8 of them (a write's pace) lie in 8
//    places modulo 128 bytes, 16 (a read's) in 16 modulo 256. And a lane's
//    accumulators hold all eight channels of c, so that it stores them as they are;
//  * dz [64 TM rows][64 p], chunk q at q ^ ((row >> 1) & 7);
//  * scales and zeros of the k-tile's rows [4 groups][64], in the forms that the
//    dequantization takes.
// A k-tile is four steps of 16 p. In steps 0 and 1 of k-tile kt the fragments of kt
// + 1 are made, from codes that were loaded a k-tile before; after step 2 the
// wavefronts meet, nobody reads the stages of kt any more, and step 3 sends dz of kt
// + 2. (A quarter of the fragments in every step, the first ones of kt + 2 and the
// loads of codes in step 3 beside dz: 631 -> 645 us for 2048 tokens, 2 of 8 experts
// 14336 -> 4096.)
// P is a multiple of 16, k-tiles of 64: the last one is the 64 rows at the end,
// with scale 0 for those that the one before has done already (an infinite dz at
// one of those: NaN, where the sum has an infinity).
//
// What bounds it: the matrix cores are busy 48% of the time (2048 tokens, 2 of 8
// experts, 14336 -> 4096: 481 GFLOP in 570 us), the fragments' instructions and
// the waits for codes and dz beside them the rest.
#include <algorithm>
#include <type_traits>

#include "expert_rows.h"
#include "paro_internal.h"
#include "w4_common.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

using namespace w4;

typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
constexpr int kRsrcWord3 = 0x00020000;  // gfx9 buffer resource word 3
constexpr int kN = 256, kM = 256, kK = 64;  // channels and rows per workgroup, k-tile

// Which chunk of fragment row r takes chunk q's place: q ^ aswap(r).
__device__ __forceinline__ int aswap(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// SHARE: dh[r] = w U[r] (fp16) and dots[2 nb + half][r], the sums over 128
// channels of U[r] h[r]; else part[r] = U[r] (fp32). The sum goes over rows p0 ..
// p0 + PP - 1 of the expert's P.
template <int TM, bool GATHER, bool SHARE>
__device__ __forceinline__ void grad_tile(const ExpertRows<GATHER>& rows_of, const ExpertTile& tile, const int nb,
                                          _Float16* A0, _Float16* A1, _Float16* B0, _Float16* B1, uint32_t* T0,
                                          uint32_t* T1, const uint8_t* __restrict__ qw,
                                          const uint16_t* __restrict__ sc, const uint8_t* __restrict__ zr,
                                          const uint16_t* __restrict__ dz, const int P, const int p0,
                                          const int PP, const int d, const int gsh, float* __restrict__ part, const uint16_t* __restrict__ h,
                                          uint16_t* __restrict__ dh) {
  constexpr int BM = 64 * TM, CB = BM / 32, NF = 4 * TM;
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, g = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = w & 1, wm = w >> 1;
  const int n0 = kN * nb, m0 = tile.first, rows = tile.end - tile.first;
  const int groups = d >> (6 + gsh), half = d >> 1;
  const size_t first = (size_t)tile.expert * P + p0;  // the first weight row
  const int KT = (PP + kK - 1) / kK;
  const __amdgpu_buffer_rsrc_t rw =
      __builtin_amdgcn_make_buffer_rsrc((void*)(qw + first * half), (short)0, PP * half, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(dz + (GATHER ? 0 : (size_t)m0 * P) + p0), (short)0,
      ((GATHER ? rows_tokens(rows_of) : rows) * P - p0) * 2, kRsrcWord3);
  // first weight row of k-tile kt (past the last one: the last again)
  auto row0 = [&](int kt) { return kt >= KT - 1 ? PP - kK : kK * kt; };

  // dz: DMA c of wavefront w fills rows 8 (CB w + c) .. + 7 (rows past the end
  // repeat the last one, never stored)
  uint32_t boff[8];
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const int r = 8 * (CB * w + c) + (lane >> 3);
    boff[c] = (uint32_t)(source_row(rows_of, m0, min(r, rows - 1)) * P + 8 * ((lane & 7) ^ ((r >> 1) & 7))) * 2u;
  }
  auto dma_b = [&](int row, _Float16* bs) {
    const int at = row * 2;
#pragma unroll
    for (int c = 0; c < CB; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)&bs[(CB * w + c) * 512], 16, boff[c], at, 0, 0);
  };

  // codes: rows 8 pr .. + 7 of the k-tile, channels n0 + 8 cb .. + 7
  const int pr = tid >> 5, cb = tid & 31;
  uint32_t coff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) coff[i] = (uint32_t)((8 * pr + i) * half + (n0 >> 1) + 4 * cb);
  struct Codes {
    uint32_t c[8];
  };
  auto load_codes = [&](int at, Codes& q) {  // at: the k-tile's first row, in bytes
#pragma unroll
    for (int i = 0; i < 8; ++i) q.c[i] = __builtin_amdgcn_raw_buffer_load_b32(rw, coff[i], at, 0);
  };
  // scale and zero: thread t has row t % 64 and group t / 64 of the channels
  // (those past the last group: the last one's, never used)
  const int trow = tid & 63, tgi = min((n0 >> (6 + gsh)) + (tid >> 6), groups - 1);
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc((void*)(sc + first * groups), (short)0, PP * groups * 2, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rz =
      __builtin_amdgcn_make_buffer_rsrc((void*)(zr + first * groups), (short)0, PP * groups, kRsrcWord3);
  const uint32_t zoff = (uint32_t)(trow * groups + tgi);
  struct Scale {
    uint32_t s, z;
  };
  auto load_scale = [&](int at, Scale& q) {  // at: the k-tile's first row, in groups
    q.s = __builtin_amdgcn_raw_buffer_load_b16(rs, 2 * zoff, 2 * at, 0);
    q.z = __builtin_amdgcn_raw_buffer_load_b8(rz, zoff, at, 0);
  };
  // scale | 1024 + z; the k-tile's first `done` rows: 0 | 1024 + z (chosen here:
  // beside the loads, the compiler waits for them there, a k-tile before)
  auto put_scale = [&](int done, const Scale& q, uint32_t* t) {
    t[tid] = (trow < done ? 0u : q.s & 0xffffu) | half_bits(1024.0f + (float)(q.z & 0xffu)) << 16;
  };
  auto done_rows = [&](int kt) { return kt >= KT - 1 ? kK * KT - PP : 0; };
  struct Rows {  // of a thread's eight rows: scale | 1024 + z
    u4 v[2];
  };

  const uint32_t one = fp16_1024_pair();
  const h2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f}, less = {(_Float16)960.0f, (_Float16)960.0f};
  const int tgroup = kK * (cb >> (3 + gsh)) + 8 * pr;
  auto get_scales = [&](const uint32_t* t, Rows& r) {
    r.v[0] = *(const u4*)(t + tgroup);
    r.v[1] = *(const u4*)(t + tgroup + 4);
  };
  // fragment of channel 8 cb + e: row arow + 32 (e / 2) + 16 (e % 2), chunk pr
  const int arow = 128 * (cb >> 4) + (cb & 15);
  const int achunk = 8 * (pr ^ aswap(cb));
  // channels 2 j and 2 j + 1
  auto fragments = [&](const Codes& q, const Rows& t, int j, _Float16* as) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t word = t.v[i >> 2][i & 3];
      const h2 sz = __builtin_bit_cast(h2, word);
      const uint32_t c = j < 2 ? q.c[i] : q.c[i] >> 8;
      h2 x;
      if (j % 2 == 0)
        x = __builtin_bit_cast(h2, (c & 0x000F000Fu) | one) - splat2(sz[1]);
      else  // (64 + z is exact)
        x = __builtin_elementwise_fma(__builtin_bit_cast(h2, (c & 0x00F000F0u) | one), sixteenth, less - splat2(sz[1]));
      v[i] = __builtin_bit_cast(uint32_t, x * splat2(sz[0]));
    }
    u4 lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], 0x05040100u);
      hi[i] = __builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], 0x07060302u);
    }
    *(u4*)(as + (arow + 32 * j) * kK + achunk) = lo;
    *(u4*)(as + (arow + 32 * j + 16) * kK + achunk) = hi;
  };

  f16v acc[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[j][i][e] = 0.0f;
  // operands of step s of a k-tile: lane half g takes chunk 4 g + s of each row
  auto read = [&](const _Float16* as, const _Float16* bs, int s, h8* a, h8* b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 32 * (4 * wn + j) + l32;
      a[j] = *(const h8*)(as + r * kK + 8 * ((4 * g + s) ^ aswap(r)));
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = 32 * (TM * wm + i) + l32;
      b[i] = *(const h8*)(bs + r * kK + 8 * ((4 * g + s) ^ ((r >> 1) & 7)));
    }
  };
  h8 a[4], b[4], an[4], bn[4];
  // a step's MFMAs on the operands in hand, among them the next step's reads, NV
  // vector instructions, NL loads and the LDS writes of two fragments
  auto step = [&](auto nv, auto nl) {
    constexpr int NV = decltype(nv)::value, NL = decltype(nl)::value;
#pragma unroll
    for (int f = 0; f < NF; ++f)
      acc[f / TM][f % TM] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[f / TM], b[f % TM], acc[f / TM][f % TM], 0, 0, 0);
    if (NL == 10) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // the scales
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (f < 4 + TM) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (NV > 0) __builtin_amdgcn_sched_group_barrier(0x002, (NV + NF - 1) / NF, 0);
      if (f < NL) {
        __builtin_amdgcn_sched_group_barrier(0x004, NV > 0 ? 1 : 2, 0);  // a load's scalar operands
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
      if (NV > 0 && f % (NF / 2) == NF / 2 - 1) __builtin_amdgcn_sched_group_barrier(0x200, 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      a[t] = an[t];
      if (t < TM) b[t] = bn[t];
    }
  };
  // s_waitcnt with lgkmcnt(0) and at most v loads still on their way
  constexpr auto wait_vm = [](int v) { return 0x70 | (v & 15) | ((v >> 4) << 14); };
  auto meet = [&](int still) {
    asm volatile("" ::: "memory");
    if (still) __builtin_amdgcn_s_waitcnt(wait_vm(10));
    else __builtin_amdgcn_s_waitcnt(wait_vm(0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  Scale szr;
  // where k-tile kt + 2 starts, and kt + 3's scales: made in the step before
  struct Ahead {
    int row, codes, scales, done;
  };
  auto ahead = [&](int kt) {
    return Ahead{row0(kt + 2), row0(kt + 2) * half, row0(kt + 3) * groups, done_rows(kt + 2)};
  };
  Ahead at = ahead(0);
  // k-tile kt in (as, bs), kt + 1's dz in bs1 and its codes in q1; fragments of
  // kt + 1 go to as1, scales of kt + 2 to the table of kt (t), codes of kt + 2 to q
  auto ktile = [&](int kt, const _Float16* as, _Float16* bs, uint32_t* t, Codes& q, _Float16* as1, const _Float16* bs1,
                   const uint32_t* t1, const Codes& q1) {
    Rows r1;
    get_scales(t1, r1);
    put_scale(at.done, szr, t);
    load_codes(at.codes, q);
    load_scale(at.scales, szr);
    read(as, bs, 1, an, bn);
    fragments(q1, r1, 0, as1);
    fragments(q1, r1, 1, as1);
    step(std::integral_constant<int, 80>{}, std::integral_constant<int, 10>{});
    read(as, bs, 2, an, bn);
    fragments(q1, r1, 2, as1);
    fragments(q1, r1, 3, as1);
    step(std::integral_constant<int, 80>{}, std::integral_constant<int, 0>{});
    read(as, bs, 3, an, bn);
    const int row = at.row;
    at = ahead(kt + 1);
    step(std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{});
    meet(1);  // still on their way: the codes of kt + 2, the scale and zero of kt + 3
    dma_b(row, bs);
    read(as1, bs1, 0, an, bn);
    step(std::integral_constant<int, 0>{}, std::integral_constant<int, CB>{});
  };

  Codes q0, q1;
  {
    Scale s0, s1;
    dma_b(row0(0), B0);
    dma_b(row0(1), B1);
    load_scale(row0(0) * groups, s0);
    load_scale(row0(1) * groups, s1);
    load_codes(row0(0) * half, q0);
    load_codes(row0(1) * half, q1);
    load_scale(row0(2) * groups, szr);
    put_scale(done_rows(0), s0, T0);
    put_scale(done_rows(1), s1, T1);
    __syncthreads();
    Rows r0;
    get_scales(T0, r0);
#pragma unroll
    for (int j = 0; j < 4; ++j) fragments(q0, r0, j, A0);
    meet(0);
    read(A0, B0, 0, a, b);
  }
  int kt = 0;
  for (; kt + 2 <= KT; kt += 2) {
    ktile(kt, A0, B0, T0, q0, A1, B1, T1, q1);
    ktile(kt + 1, A1, B1, T1, q1, A0, B0, T0, q0);
  }
  if (kt < KT) ktile(kt, A0, B0, T0, q0, A1, B1, T1, q1);
  __builtin_amdgcn_s_waitcnt(wait_vm(0));  // (the last DMA lands before the workgroup's LDS is another's)

  // acc[j][i][4 q + c] = U[m0 + 32 (TM wm + i) + l32][channel 8 (16 (nb 2 + wn) + 8 (q % 2) + 4 g + c) + 2 j + q / 2]
  const int nw0 = n0 + 128 * wn;
  auto channel = [&](int x) { return nw0 + 8 * (8 * (x >> 2) + 4 * g + (x & 3)); };
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = m0 + 32 * (TM * wm + i) + l32;
    if constexpr (SHARE) {
      float dot = 0.0f;
      if (m < tile.end) {
        const float share = rows_of.weight(m);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int qb = x >> 2, c = x & 3, ch = channel(x);
          if (ch < d) {
            const u4 hv = *(const u4*)(h + (size_t)m * d + ch);
            u4 o;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float u0 = acc[e >> 1][i][4 * qb + c], u1 = acc[e >> 1][i][4 * (2 + qb) + c];
              const uint32_t hw = hv[e >> 1];
              dot = __builtin_fmaf(u0, half_lo(hw), dot);
              dot = __builtin_fmaf(u1, half_hi(hw), dot);
              o[e >> 1] = half_bits(u0 * share) | (half_bits(u1 * share) << 16);
            }
            *(u4*)(dh + (size_t)m * d + ch) = o;
          }
        }
      }
      dot += __shfl_xor(dot, 32);
      if (g == 0 && m < tile.end) part[(size_t)(2 * nb + wn) * rows_of.t.R + m] = dot;
    } else {
      if (m < tile.end) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int qb = x >> 2, c = x & 3, ch = channel(x);
          if (ch < d) {
            float* o = part + (size_t)m * d + ch;
#pragma unroll
            for (int e = 0; e < 8; e += 4)
              *(f4*)(o + e) = f4{acc[e >> 1][i][4 * qb + c], acc[e >> 1][i][4 * (2 + qb) + c],
                                 acc[(e >> 1) + 1][i][4 * qb + c], acc[(e >> 1) + 1][i][4 * (2 + qb) + c]};
          }
        }
      }
    }
  }
}

// Tiles of up to 256 rows. An expert's last one may be short: up to 128 rows in
// wavefront tiles of half the height, which take 0.6 of a whole tile's time. Where
// there are few tiles, `splits` workgroups share out a tile's sum (sums in part
// [splits][R][d]).
template <bool GATHER, bool SHARE>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1)))
void experts_grad_kernel(ExpertRows<GATHER> rows_of, const uint8_t* __restrict__ qw, const uint16_t* __restrict__ sc,
                         const uint8_t* __restrict__ zr, const uint16_t* __restrict__ dz, int P, int d, int gsh,
                         int nblk, int splits, float* __restrict__ part, const uint16_t* __restrict__ h,
                         uint16_t* __restrict__ dh) {
  __shared__ __attribute__((aligned(1024))) _Float16 A0[kN * kK], A1[kN * kK], B0[kM * kK], B1[kM * kK];
  __shared__ __attribute__((aligned(16))) uint32_t T0[4 * kK], T1[4 * kK];
  ExpertTile tile;
  int nb;
  int b = blockIdx.x, p0 = 0, PP = P;
  if constexpr (!SHARE) {
    const int per = gridDim.x / splits, sp = b / per, KT = (P + kK - 1) / kK;
    b -= sp * per;
    p0 = kK * (int)((int64_t)KT * sp / splits);
    PP = (sp + 1 == splits ? P : kK * (int)((int64_t)KT * (sp + 1) / splits)) - p0;
    part += (size_t)sp * rows_of.t.R * d;
  }
  if (!rows_of.find_tile_halves(b, kM, nblk, tile, nb)) return;
  if (tile.end - tile.first > kM / 2)
    grad_tile<4, GATHER, SHARE>(rows_of, tile, nb, A0, A1, B0, B1, T0, T1, qw, sc, zr, dz, P, p0, PP, d, gsh, part, h,
                                  dh);
  else
    grad_tile<2, GATHER, SHARE>(rows_of, tile, nb, A0, A1, B0, B1, T0, T1, qw, sc, zr, dz, P, p0, PP, d, gsh, part, h,
                                  dh);
}

template <bool GATHER, bool SHARE>
hipError_t launch(const ExpertRouting& t, const uint16_t* dz, const uint8_t* qweight, const uint16_t* scales,
                  const uint8_t* zeros, int64_t P, int64_t d, int group, int splits, float* part, const uint16_t* h,
                  uint16_t* dh, hipStream_t stream) {
  const int gsh = group == 64 ? 0 : group == 128 ? 1 : 2;
  const unsigned nblk = (unsigned)((d + kN - 1) / kN);
  const unsigned tiles = nblk * (unsigned)expert_blocks(t, kM);
  hipLaunchKernelGGL((experts_grad_kernel<GATHER, SHARE>), dim3(((tiles + 7) / 8 * 8 + 8) * (unsigned)splits), dim3(256), 0, stream,
                     ExpertRows<GATHER>{t}, qweight, scales, zeros, dz, (int)P, (int)d, gsh, (int)nblk, splits,
                     part, h, dh);
  return hipGetLastError();
}

}  // namespace

// Workgroups that share a tile's sum over P rows, at least 16 k-tiles each: as many as
// make one and a half tiles a CU. (gated 4096 -> 14336, 8 experts, one workgroup a tile
// | three: a mean of 128 rows 727 | 424 us, 192 718 | 537.)
int experts_grad_splits(const ExpertRouting& t, int64_t P, int64_t d) {
  const int64_t blocks = std::max<int64_t>(std::min<int64_t>(t.E, t.R), t.R / kM) * ((d + kN - 1) / kN);
  return (int)std::max<int64_t>(1, std::min<int64_t>({384 / blocks, P / (16 * kK), 4}));
}

void experts_grad_wide_steps(int64_t E, int64_t d, std::vector<int64_t>& rows) {
  rows.insert(rows.end(), {E, 16 * E - 1, 160 * E - 1});
  for (int64_t s = 1; s <= 4; ++s) {
    const int64_t q = 384 / s / ((d + kN - 1) / kN);
    rows.insert(rows.end(), {q, kM * (q + 1) - 1});
  }
}

// Whether the gradient is taken in these tiles (share: of combine, whose tiles are not
// shared out), from a mean of 16 rows on if there are tiles for all CUs, else of 160.
// Microseconds of w4_input_grad_rows_kernel's way | this:
//   of 2048 -> 1024, 64 experts: a mean of 8 rows 47 | 46, 16: 55 | 48, 64: 107 | 67;
//   of gated 1408 -> 2048, 60 experts: 16: 151 | 172, 48: 225 | 242, 96: 395 | 356;
//   of 14336 <- 4096, 8 experts (128 tiles): 32: 164 | 200, 128: 266 | 312, 192: 370 | 321;
//   of gated 4096 -> 14336, 8 experts (128 tiles, shared out), dz included: 16: 469 | 476,
//     32: 532 | 513, 64: 626 | 551, 128: 966 | 793.
// (The rule goes by rows and tiles: with 60 experts of 1408 -> 2048 it is wrong up to
// some 50 rows, by 14% at 16.)
bool experts_grad_wide_fit(const ExpertRouting& t, int64_t P, int64_t d, bool share) {
  const int64_t E = t.E, splits = share ? 1 : experts_grad_splits(t, P, d);
  return P >= kK && t.R >= (E * d * splits >= kN * 256 ? 16 : 160) * E;
}

// partial dots of the weights' gradients: [2 ceil(d / 256)][R]
size_t experts_grad_dots(const ExpertRouting& t, int64_t d) { return (size_t)((d + kN - 1) / kN) * 2 * t.R * 4; }

hipError_t launch_w4_experts_grad_part(const ExpertRouting& t, const uint16_t* dz, const uint8_t* qweight,
                                       const uint16_t* scales, const uint8_t* zeros, float* part, int64_t P, int64_t d,
                                       int group, hipStream_t stream) {
  return launch<false, false>(t, dz, qweight, scales, zeros, P, d, group, experts_grad_splits(t, P, d), part, nullptr,
                              nullptr, stream);
}

hipError_t launch_w4_experts_grad_share(const ExpertRouting& t, const uint16_t* dy, const uint8_t* qweight,
                                        const uint16_t* scales, const uint8_t* zeros, float* dots, const uint16_t* h,
                                        uint16_t* dh, int64_t P, int64_t d, int group, hipStream_t stream) {
  return launch<true, true>(t, dy, qweight, scales, zeros, P, d, group, 1, dots, h, dh, stream);
}

}  // namespace paro
