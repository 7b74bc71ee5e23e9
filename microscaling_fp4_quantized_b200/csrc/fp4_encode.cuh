// The microscaling FP4 block rule: the E4M3 scale byte of 16 elements and their E2M1 codes,
// shared by the attention quantizer and the paged cache.
#pragma once

#include <cstdint>

#include "sm100_ptx.cuh"

namespace sage {

// x / d rounded to nearest even, from r = RN(1/d): the FMA-corrected quotient of
// Markstein ("IA-64 and Elementary Functions: Speed and Precision", 2000, ch. 8):
// q = RN(x r), e = x - q d (exact with an FMA), result RN(q + e r). It is not correctly
// rounded for every divisor, so it is used only where it was checked exhaustively on the
// CPU against IEEE binary32 division: d = any positive E4M3 value with |x/d| in
// [2^-4, 2^4) (E2M1 codes outside that range do not depend on the last bit of the
// quotient), and d = 6 for every positive binary32 x with a normal quotient (a subnormal
// a/6 gives scale byte 0 either way). The sign is copied from x so that -0 / d = -0.
__device__ __forceinline__ float div_fma(float x, float d, float r) {
  const float q = __fmul_rn(x, r);
  const float e = __fmaf_rn(-q, d, x);
  return copysignf(__fmaf_rn(e, r, q), x);
}

// RN(1/6) in binary32.
constexpr float kRecip6 = 0.16666667163372039794921875f;

// E4M3 scale byte of a block with maximum magnitude a: E4M3(RN(a / 6)).
__device__ __forceinline__ uint32_t block_scale_byte(float a) {
  return f32_to_e4m3(div_fma(a, 6.0f, kRecip6));
}

// Codes of 8 values (x[O .. O + 7]) against a decoded scale s (s == 0 -> zero codes);
// element O lands in the low nibble of the low byte. Each code is E2M1(RN(x / s)) with
// RN(x / s) formed as div_fma does, two lanes per instruction and with the reciprocal
// negated: q' = RN(x * -r) = -RN(x r); e = RN(x + q' s) = x - RN(x r) s, div_fma's exact
// remainder; RN(e * -r + q') = -RN(e r + RN(x r)). Rounding to nearest is symmetric, so
// every lane holds exactly -div_fma(x, s, r) -- and, for x = +-0 or a product that
// underflows, the zero of the sign opposite to x's, i.e. minus div_fma's copysign result.
// E2M1 rounding is symmetric too, so the codes come out with every sign bit inverted,
// which one XOR puts back. (Checked on the CPU for every E4M3 divisor and every finite
// quotient tried, +-0 and underflowing products included: tests/div_identity.c.)
//
// r = RN(1/s) for a positive E4M3 s: the approximate reciprocal is off by e, |e| <= 2^-23 or so; 1 - s r0 = e is exact
// in the FMA (s has 4 significant bits), and r0 + r0 e = (1 - e^2) / s is rounded once. 1/s times its power of two is
// 1, 8/9, 4/5, 8/11, 2/3, 8/13, 4/7 or 8/15, whose binary periods of at most 12 places keep it further than 2^-46
// from every rounding border, so the result is the correctly rounded one.
template <int O, int N>
__device__ __forceinline__ uint32_t encode8_neg(const float (&x)[N], float s) {
  if (s == 0.0f) return 0u;
  float r0;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(s));
  const float nr = -__fmaf_rn(r0, __fmaf_rn(-s, r0, 1.0f), r0);
  const float2 nr2 = make_float2(nr, nr), s2 = make_float2(s, s);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 xv = make_float2(x[O + 2 * i], x[O + 2 * i + 1]);
    const float2 nq = mul2(xv, nr2);
    const float2 e = fma2(nq, s2, xv);
    const float2 r = fma2(e, nr2, nq);
    y[2 * i] = r.x;
    y[2 * i + 1] = r.y;
  }
  return f32x8_to_e2m1(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]) ^ 0x88888888u;
}

}  // namespace sage
