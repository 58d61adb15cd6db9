// The activations of the gates (rapt_act in include/rapt.h) and their derivatives, in fp32, for the
// residual norm and the gated feed-forward.
#pragma once

#include <stdint.h>

namespace rapt {

enum class Act { None = 0, Silu = 1, Gelu = 2, Relu = 3, Sigmoid = 4 };

// 1 / (1 + e^-z) from the hardware's 2^x and 1/x. The rounding of z log2(e) puts e^-z off by 1.5 |z| 2^-24 of
// itself beside the 2^-22 of 2^x. e^-z overflows to infinity below z = -88; the quotient is then an exact 0.
__device__ __forceinline__ float sigmoid_f(float z) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}
// The same for a derivative, and e = e^-z: 1 - s is formed as e s, which keeps its bits where s is near one
// (as a difference it has lost 6 % at z = 16). The exponent stops at 2^127, where s is 0 as well, so that e s is
// no infinity times zero; a NaN passes.
__device__ __forceinline__ float sigmoid_f(float z, float& e) {
  float w, s;
  asm("min.NaN.f32 %0, %1, 0f42FE0000;" : "=f"(w) : "f"(z * -1.4426950408889634f));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(w));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// The normal distribution function Phi(z), and e^(-z^2 / 2). With x = |z| / sqrt(2), Abramowitz and
// Stegun's formula 7.1.26 gives erfc(x) = (a1 t + ... + a5 t^5) e^(-x^2), t = 1 / (1 + p x), within
// 1.5e-7, and Phi(-|z|) is half of that: the exponential is the one that the derivative needs.
__device__ __forceinline__ float phi_f(float z, float& bell) {
  const float x = fabsf(z) * 0.70710678118654752f;
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3275911f, x, 1.f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(bell) : "f"(x * x * -1.4426950408889634f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float tail = 0.5f * q * t * bell;
  return z < 0.f ? tail : 1.f - tail;
}

// gelu(z) = z Phi(z) and, where GRAD, its derivative Phi(z) + z phi(z) for two values at once: the steps of
// phi_f with two fp32 values per instruction, and the same bits.
template <bool GRAD>
__device__ __forceinline__ void gelu_two(float2 z, float2& a, float2& da) {
  const auto both = [](float v) { return make_float2(v, v); };
  const float2 x = __fmul2_rn(make_float2(fabsf(z.x), fabsf(z.y)), both(0.70710678118654752f));
  const float2 u = __ffma2_rn(both(0.3275911f), x, both(1.f));
  const float2 w = __fmul2_rn(__fmul2_rn(x, x), both(-1.4426950408889634f));
  float2 t, bell;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(u.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(u.y));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(bell.x) : "f"(w.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(bell.y) : "f"(w.y));
  float2 q = __ffma2_rn(both(1.061405429f), t, both(-1.453152027f));
  q = __ffma2_rn(q, t, both(1.421413741f));
  q = __ffma2_rn(q, t, both(-0.284496736f));
  q = __ffma2_rn(q, t, both(0.254829592f));
  const float2 tail = __fmul2_rn(__fmul2_rn(__fmul2_rn(both(0.5f), q), t), bell);
  const float2 rest = __ffma2_rn(tail, both(-1.f), both(1.f));
  const float2 cdf = make_float2(z.x < 0.f ? tail.x : rest.x, z.y < 0.f ? tail.y : rest.y);
  a = __fmul2_rn(z, cdf);
  if (GRAD) da = __ffma2_rn(__fmul2_rn(z, both(0.39894228040143268f)), bell, cdf);
}

// act(z), and act'(z) where GRAD. relu'(0) = 0.
template <bool GRAD>
__device__ __forceinline__ void act_one(Act act, float z, float& a, float& da) {
  switch (act) {
    case Act::None:
      a = z;
      if (GRAD) da = 1.f;
      break;
    case Act::Relu:
      a = z <= 0.f ? 0.f : z;  // a NaN stays one
      if (GRAD) da = z > 0.f ? 1.f : 0.f;
      break;
    case Act::Gelu: {  // z Phi(z); derivative Phi(z) + z phi(z)
      float bell;
      const float cdf = phi_f(z, bell);
      a = z * cdf;
      if (GRAD) da = fmaf(z * 0.39894228040143268f, bell, cdf);
      break;
    }
    case Act::Sigmoid: {
      float e;
      const float s = GRAD ? sigmoid_f(z, e) : sigmoid_f(z);
      a = s;
      if (GRAD) da = s * (e * s);
      break;
    }
    case Act::Silu: {
      float e;
      const float s = GRAD ? sigmoid_f(z, e) : sigmoid_f(z);
      a = z * s;
      if (GRAD) da = s * fmaf(z, e * s, 1.f);
      break;
    }
  }
}

// The same over N values: the (uniform) choice is made once, outside the loop.
template <int N, bool GRAD>
__device__ __forceinline__ void act_vec(Act act, const float (&z)[N], float (&a)[N], float (&da)[N]) {
#define RAPT_ACT_CASE(X)                                        \
  case Act::X:                                                  \
    _Pragma("unroll") for (int i = 0; i < N; ++i) act_one<GRAD>(Act::X, z[i], a[i], da[i]); \
    break;
  switch (act) {
    RAPT_ACT_CASE(None)
    RAPT_ACT_CASE(Silu)
    case Act::Gelu:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float2 p, d;
        gelu_two<GRAD>(make_float2(z[i], z[i + 1]), p, d);
        a[i] = p.x;
        a[i + 1] = p.y;
        if (GRAD) da[i] = d.x, da[i + 1] = d.y;
      }
      break;
    RAPT_ACT_CASE(Relu)
    RAPT_ACT_CASE(Sigmoid)
  }
#undef RAPT_ACT_CASE
}

}  // namespace rapt
