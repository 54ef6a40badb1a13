// Epilogues of the W4 products: what becomes of Z = X' W_hat^T (fp32) before
// it is rounded to fp16.
//   kEpiPlain      y = Z + b
//   kEpiAct        y = act(Z + b) + R
//   kEpiGated      y = act(Zg + bg) (Zu + bu), Zg and Zu the first and the
//                  second N rows of the weight block
//   kEpiActGrad    dz = dy act'(Z + b)
//   kEpiGatedGrad  dzg = dy (Zu + bu) act'(Zg + bg), dzu = dy act(Zg + bg)
//   kEpiShare      y = w (Z + b), w a row's own weight, fp32 (a token's experts
//                  are summed from these)
// All in fp32 with one rounding to fp16 at the store (kEpiShare: none).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/paro.h"
#include "w4_common.h"

namespace paro {

enum { kEpiPlain = 0, kEpiAct = 1, kEpiGated = 2, kEpiActGrad = 3, kEpiGatedGrad = 4, kEpiShare = 5 };
constexpr bool epi_gated(int epi) { return epi == kEpiGated || epi == kEpiGatedGrad; }

// The activation as the kernels take it: silu and gelu_tanh are both
// z * sigmoid(u), u = z (a + b z^2) (tanh(t) = 2 sigmoid(2 t) - 1), so one
// instruction sequence with two coefficients covers them, and none and relu
// are selected from it; the erf form is compiled separately (ERF).
struct ActForm {
  float a, b;
  int kind;  // 0 none, 1 z sigmoid(u), 2 relu
};

inline ActForm act_form(int32_t act) {
  constexpr float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  switch (act) {
    case PARO_ACT_SILU: return {1.0f, 0.0f, 1};
    case PARO_ACT_GELU_TANH: return {c, c * 0.044715f, 1};
    case PARO_ACT_RELU: return {0.0f, 0.0f, 2};
    default: return {0.0f, 0.0f, 0};
  }
}

namespace w4 {

// sigmoid(u): exp2 and rcp of the hardware, each within an ulp or two of
// fp32, two thousand times finer than the fp16 rounding of the result
__device__ __forceinline__ float sigmoid(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * u));
}

// The normal distribution function Phi(z) = erfc(-z / sqrt 2) / 2 of the erf
// gelu, and e = exp(-z^2 / 2): for x = |z| / sqrt 2, erfc(x) = exp(-x^2) t P(t)
// with t = 1 / (1 + 0.425 x) and P a polynomial of degree 7 fitted in relative
// terms. The fit is off by at most 4.5e-7 of Phi for |z| <= 8 (1.8e-6 to |z| =
// 17); evaluated in fp32, where the rounding of exp2's argument adds about
// 2^-24 z^2, Phi(-|z|) is off by 5.8e-7 to |z| = 1, 7.4e-7 to 3, 1.5e-6 to 5
// and 3.0e-6 to 8: less than a hundredth of an fp16 rounding (4.9e-4) down to
// where z Phi(z) is no fp16 number any more (z = -5.7). The math library's
// erfc took 2.3 us more of a 333 x 2560 -> 1040 call.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.425f * 0.7071067811865476f * __builtin_fabsf(z));
  float p = 0.0688890740275383f;
  p = __builtin_fmaf(p, t, -0.3024859130382538f);
  p = __builtin_fmaf(p, t, 0.38947463035583496f);
  p = __builtin_fmaf(p, t, -0.08682318031787872f);
  p = __builtin_fmaf(p, t, 0.2465682476758957f);
  p = __builtin_fmaf(p, t, 0.20322471857070923f);
  p = __builtin_fmaf(p, t, 0.24144889414310455f);
  p = __builtin_fmaf(p, t, 0.23970328271389008f);
  e = __builtin_amdgcn_exp2f(-0.7213475204444817f * z * z);
  const float q = 0.5f * e * t * p;
  return z < 0.0f ? q : 1.0f - q;
}

// u of act_form. The square's term is held finite: with b = 0 an infinite z
// would make it NaN, and silu(+inf) is +inf.
__device__ __forceinline__ float act_argument(float z, const ActForm& f) {
  return z * (f.a + __builtin_fminf(f.b * z * z, 3.402823466e+38f));
}

// (a NaN passes through every form: the relu keeps what is not below zero)
template <bool ERF>
__device__ __forceinline__ float act_value(float z, const ActForm& f) {
  float e;
  if constexpr (ERF) return z * normal_cdf(z, e);
  const float s = z * sigmoid(act_argument(z, f));
  const float r = z < 0.0f ? 0.0f : z;
  return f.kind == 1 ? s : f.kind == 2 ? r : z;
}

// act(z) and act'(z)
template <bool ERF>
__device__ __forceinline__ void act_both(float z, const ActForm& f, float& v, float& dv) {
  if constexpr (ERF) {
    float e;
    const float phi = normal_cdf(z, e);
    v = z * phi;
    dv = phi + z * 0.3989422804014327f * e;
  } else {
    const float s = sigmoid(act_argument(z, f));
    const float sv = z * s;
    const float sd = s + sv * (1.0f - s) * (f.a + 3.0f * f.b * z * z);
    const float r = z < 0.0f ? 0.0f : z;
    v = f.kind == 1 ? sv : f.kind == 2 ? r : z;
    dv = f.kind == 1 ? sd : f.kind == 2 ? (z > 0.0f ? 1.0f : 0.0f) : 1.0f;
  }
}

// Epilogue of one block of a wavefront's outputs: 64 tokens (rows m0 .. + 63)
// by NJ tiles of 32 weight rows, get(j, t, e) = Z of tile j, token 32 t +
// lane % 32, tile row 8 (e / 4) + 4 (lane / 32) + e % 4. Plain weight rows are
// output channels c0 + 32 j + ...; gated blocks interleave gate and up rows in
// runs of eight (tile row r: channel 8 (r / 16) + r % 8, up when (r / 8) is
// odd), so a lane holds both halves of its 16 NJ channels from c0 on.
// epi_fetch loads the block's rows of the second operand (residual or dy) into
// registers, which the caller does ahead of the block, so that their way from
// memory overlaps what comes before.
// `stage` is this wavefront's own 64 x 32 NJ halfs of LDS: the second operand
// comes in and the results go out through it as whole rows
// (16-byte chunk c of row r at c ^ (r % chunks)), and the lane that reads an
// element of the second operand replaces it in place by the result, so no
// rounding happens in between. Its LDS accesses complete in order, so no
// barrier is needed. y may be aux (every element is read before it is
// written, by the same wavefront).
template <int EPI>
__device__ __forceinline__ bool epi_has_aux(const uint16_t* aux) {
  return EPI == kEpiAct ? aux != nullptr : EPI == kEpiActGrad || EPI == kEpiGatedGrad;
}
template <int EPI, int NJ>
__device__ __forceinline__ void epi_fetch(u4* av, int lane, int m0, int c0, int M, int N, const uint16_t* aux) {
  constexpr int CO = epi_gated(EPI) ? 2 * NJ : 4 * NJ;
  if (!epi_has_aux<EPI>(aux)) return;
#pragma unroll
  for (int rr = 0; rr < CO; ++rr) {
    const int m = m0 + (64 / CO) * rr + lane / CO, n = c0 + 8 * (lane % CO);
    av[rr] = u4{0u, 0u, 0u, 0u};
    if (m < M && n < N) av[rr] = *(const u4*)(aux + (size_t)m * N + n);
  }
}
template <int EPI, int NJ, bool ERF, class Get>
__device__ __forceinline__ void epi_block(uint8_t* stage, Get get, const u4* av, int lane, int m0, int c0, int M,
                                          int N, const uint16_t* bias, const uint16_t* aux, const ActForm& act,
                                          uint16_t* y) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  constexpr bool GT = epi_gated(EPI);
  constexpr int CO = GT ? 2 * NJ : 4 * NJ;               // chunks of 8 output channels per token
  constexpr int CR = EPI == kEpiGatedGrad ? 2 * CO : CO;  // chunks per staged row (dzg, then dzu)
  constexpr int RB = 16 * CR;
  const int l32 = lane & 31, g = lane >> 5;
  auto at = [&](int row, int chunk) { return stage + row * RB + ((chunk ^ (row % CR)) << 4); };
  auto half4 = [](u2 v, float* o) {
    o[0] = half_lo(v[0]);
    o[1] = half_hi(v[0]);
    o[2] = half_lo(v[1]);
    o[3] = half_hi(v[1]);
  };
  auto pack4 = [](const float* o) {
    return u2{half_bits(o[0]) | (half_bits(o[1]) << 16), half_bits(o[2]) | (half_bits(o[3]) << 16)};
  };
  const bool has_aux = epi_has_aux<EPI>(aux);
  if (has_aux) {
#pragma unroll
    for (int rr = 0; rr < CO; ++rr) *(u4*)at((64 / CO) * rr + lane / CO, lane % CO) = av[rr];
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int q = 0; q < 4; q += GT ? 2 : 1) {
      // first of the lane's four channels inside the block
      const int nl = GT ? 16 * j + 4 * q + 4 * g : 32 * j + 8 * q + 4 * g;
      float b0[4] = {0.f, 0.f, 0.f, 0.f}, b1[4] = {0.f, 0.f, 0.f, 0.f};
      if (bias && c0 + nl < N) {
        half4(*(const u2*)(bias + c0 + nl), b0);
        if constexpr (GT) half4(*(const u2*)(bias + N + c0 + nl), b1);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int rl = 32 * t + l32;
        u2* p0 = (u2*)(at(rl, nl >> 3) + (((nl >> 2) & 1) << 3));
        float o0[4], o1[4], a4[4] = {0.f, 0.f, 0.f, 0.f};
        if (has_aux) half4(*p0, a4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float z0 = get(j, t, 4 * q + c) + b0[c];
          if constexpr (EPI == kEpiAct) {
            o0[c] = act_value<ERF>(z0, act) + a4[c];
          } else if constexpr (EPI == kEpiActGrad) {
            float v, dv;
            act_both<ERF>(z0, act, v, dv);
            o0[c] = a4[c] * dv;
          } else {
            const float z1 = get(j, t, 4 * (q + 1) + c) + b1[c];
            if constexpr (EPI == kEpiGated) {
              o0[c] = act_value<ERF>(z0, act) * z1;
            } else {
              float v, dv;
              act_both<ERF>(z0, act, v, dv);
              o0[c] = a4[c] * z1 * dv;
              o1[c] = a4[c] * v;
            }
          }
        }
        *p0 = pack4(o0);
        if constexpr (EPI == kEpiGatedGrad) *(u2*)(at(rl, CO + (nl >> 3)) + (((nl >> 2) & 1) << 3)) = pack4(o1);
      }
    }
  }
#pragma unroll
  for (int rr = 0; rr < CR; ++rr) {
    const int rl = (64 / CR) * rr + lane / CR, c = lane % CR;
    const u4 v = *(const u4*)at(rl, c);
    const int m = m0 + rl, n = c0 + 8 * (c % CO);
    if (m < M && n < N) {
      if constexpr (EPI == kEpiGatedGrad) *(u4*)(y + ((size_t)m * 2 + c / CO) * N + n) = v;
      else *(u4*)(y + (size_t)m * N + n) = v;
    }
  }
}

// Epilogue of four neighbouring channels of one token held by one lane: from
// the sums z[0] of channels n .. n + 3 (gated: the gate's, and z[1] the up
// projection's) to the output. y may be aux.
template <int EPI>
__device__ __forceinline__ void epi_lane(f4* z, int m, int n, int N, const uint16_t* bias, const uint16_t* aux,
                                         const ActForm& act, int erf, uint16_t* y) {
  auto read4 = [](const uint16_t* p) {
    const uint2 raw = *(const uint2*)p;
    return f4{half_lo(raw.x), half_hi(raw.x), half_lo(raw.y), half_hi(raw.y)};
  };
  auto write4 = [](uint16_t* p, const f4& v) {
    uint2 o;
    o.x = half_bits(v[0]) | (half_bits(v[1]) << 16);
    o.y = half_bits(v[2]) | (half_bits(v[3]) << 16);
    *(uint2*)p = o;
  };
  if (bias) {
    z[0] += read4(bias + n);
    if constexpr (epi_gated(EPI)) z[1] += read4(bias + N + n);
  }
  if constexpr (EPI == kEpiAct || EPI == kEpiGated) {
#pragma unroll
    for (int e = 0; e < 4; ++e) z[0][e] = erf ? act_value<true>(z[0][e], act) : act_value<false>(z[0][e], act);
    if constexpr (EPI == kEpiGated) z[0] *= z[1];
    else if (aux) z[0] += read4(aux + (size_t)m * N + n);
    write4(y + (size_t)m * N + n, z[0]);
  } else {
    const f4 dy = read4(aux + (size_t)m * N + n);
    f4 v, dv;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      if (erf) act_both<true>(z[0][e], act, a, b);
      else act_both<false>(z[0][e], act, a, b);
      v[e] = a;
      dv[e] = b;
    }
    if constexpr (EPI == kEpiActGrad) {
      write4(y + (size_t)m * N + n, dy * dv);
    } else {
      write4(y + (size_t)m * 2 * N + n, dy * z[1] * dv);
      write4(y + ((size_t)m * 2 + 1) * N + n, dy * v);
    }
  }
}

// kEpiShare of four neighbouring channels of one row held by one lane.
__device__ __forceinline__ void epi_share(f4 z, float weight, int m, int n, int N, const uint16_t* bias, float* y) {
  if (bias) {
    const uint2 raw = *(const uint2*)(bias + n);
    z += f4{half_lo(raw.x), half_hi(raw.x), half_lo(raw.y), half_hi(raw.y)};
  }
  *(f4*)(y + (size_t)m * N + n) = z * weight;
}

}  // namespace w4
}  // namespace paro
