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

// gelu(z) = z Phi(z) (Phi the normal distribution function) and, where GRAD, its derivative Phi(z) + z phi(z),
// for two values at once, two fp32 values an instruction.
//
// With a = |z| and s = a / (1 + 0.335 a), Phi(-a) e^(a^2 / 2) is 1/2 plus s times a polynomial of s, fitted here
// to scipy's erfcx(a / sqrt(2)) / 2 over [0, 13.3] by weighted least squares made minimax: within
// 6.3e-8 (1 + a^2 / 3) of its own value. So the left tail keeps its relative accuracy (a formula with an
// absolute bound has lost 1 % of Phi at z = -8), and near 0, where s is small, the roundings of 1/x and s
// hardly count. The exponential, off by 1.25 a^2 2^-24 and the 2^-22 of the hardware's 2^x, is the one that
// phi needs. Beyond a = 16 it is 0, where a stops so that an infinity is not multiplied with it.
template <bool GRAD>
__device__ __forceinline__ void gelu_two(float2 z, float2& a, float2& da) {
  const auto both = [](float v) { return make_float2(v, v); };
  const float2 x = make_float2(fminf(fabsf(z.x), 16.f), fminf(fabsf(z.y), 16.f));
  const float2 u = __ffma2_rn(both(0.335f), x, both(1.f));
  const float2 w = __fmul2_rn(__fmul2_rn(x, x), both(-0.72134752044448170f));
  float2 t, bell;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(u.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(u.y));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(bell.x) : "f"(w.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(bell.y) : "f"(w.y));
  const float2 s = __fmul2_rn(x, t);
  float2 q = __ffma2_rn(both(-2.25599924e-05f), s, both(0.000157447837f));
  q = __ffma2_rn(q, s, both(5.16042201e-05f));
  q = __ffma2_rn(q, s, both(-0.00186502805f));
  q = __ffma2_rn(q, s, both(-0.0103010526f));
  q = __ffma2_rn(q, s, both(0.1163643f));
  q = __ffma2_rn(q, s, both(-0.398942888f));
  q = __ffma2_rn(q, s, both(0.5f));
  const float2 tail = __fmul2_rn(q, bell);
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
    case Act::Gelu: {
      float2 p, d;
      gelu_two<GRAD>(make_float2(z, z), p, d);
      a = p.x;
      if (GRAD) da = d.x;
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
