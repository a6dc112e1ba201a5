// 16- and 32-bit values as 8-bit codes of an exact quotient (rounded to nearest, ties to even): what the cache write and the
// block quantisation share.
#pragma once
#include "attn.h"

namespace sffn {

// max over aligned groups of G lanes
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if (G >= 2) v = max(v, dpp_u<0xB1>(v));
  if (G >= 4) v = max(v, dpp_u<0x4E>(v));
  if (G >= 8) v = max(v, dpp_u<0x141>(v));
  if (G >= 16) v = max(v, dpp_u<0x140>(v));
  if (G >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, WAVE));
  return v;
}

// b / TOP, correctly rounded (shown for every mantissa of 11 bits by exact arithmetic; below 2^-60 it does not matter)
template <int TOP>
__device__ __forceinline__ float over_top(float b) {
  constexpr float R = 1.f / TOP;
  const float q = b * R;
  return fmaf(fmaf(-q, (float)TOP, b), R, q);
}

// four codes of x * f, rounded to nearest even
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(const float* x, float f) {
  if constexpr (E4M3) {
    const int u = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * f, x[1] * f, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * f, x[3] * f, u, true);
  } else {
    uint32_t b[4];                                           // x f + 1.5 * 2^23 has the rounded x f in its low byte
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(x[i], f, 12582912.f));
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u),
                                 __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), 0x05040100u);
  }
}
// A value that rounds to the same code as the exact quotient x / s. inv: 1 / s to within a few steps. A code or the middle
// between two of them has at most 5 significant bits (e4m3) or is a multiple of 1/2 (int8): h is the one nearest to the
// quotient, and the sign of the remainder x - h s (one rounding: exact) tells on which side of it the quotient lies.
template <bool E4M3>
__device__ __forceinline__ float beside(float x, float s, float inv) {
  const float h = E4M3 ? __uint_as_float((__float_as_uint(x * inv) + 0x40000u) & 0xFFF80000u)
                       : fmaf(x, inv, 6291456.f) - 6291456.f;      // 1.5 * 2^22: steps of 1/2
  constexpr float T = E4M3 ? 0x1p-15f : 0x1p-8f;   // 2^-15 is one step at 448; what is nearer to 0 than 2^-10 is 0
  return h + __builtin_amdgcn_fmed3f(fmaf(-h, s, x) * 0x1p100f, -T, T);
}
// Codes of x[0 .. 8) / s, rounded to nearest even from the exact quotients. 1 / s lies between two fp32 factors; where
// both give the same codes, these are the quotients' codes, else (in one of the wave's rows) remainders decide. A value
// with the largest one's mantissa is a middle or within a step of one, which every second wave of bf16 rows holds: those
// go to the remainders at once (4000 tokens of 40 heads of 128, bf16 to e4m3: 31.9 -> 30.0 us; 3300 from fp16 to int8:
// with the factors 21.2 us, without 22.6). Quotients are at most top (1 + 2^-23) by the scale's making: nothing needs a
// limit.
template <bool E4M3, bool BF>
__device__ __forceinline__ uint2 encode8(const float* x, float s) {
  const float inv = __builtin_amdgcn_rcpf(s);
  uint2 c = make_uint2(0, 0);
  bool same = false;
  if constexpr (!BF) {
    const float lo = inv * (1.f - 0x1p-20f), hi = inv * (1.f + 0x1p-20f);
    c = make_uint2(encode4<E4M3>(x, lo), encode4<E4M3>(x + 4, lo));
    same = !__any(((c.x ^ encode4<E4M3>(x, hi)) | (c.y ^ encode4<E4M3>(x + 4, hi))) != 0);
  }
  if (!same) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = beside<E4M3>(x[i], s, inv);
    c = make_uint2(encode4<E4M3>(q, 1.f), encode4<E4M3>(q + 4, 1.f));
  }
  return c;
}

}  // namespace sffn
