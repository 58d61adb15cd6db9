// The activations of the gates (rapt_act in include/rapt.h) and their derivatives, in fp32, for the
// residual norm and the gated feed-forward.
#pragma once

#include <stdint.h>

namespace rapt {

enum class Act { None = 0, Silu = 1, Gelu = 2, Relu = 3, Sigmoid = 4 };

// 1 / (1 + e^-z), both to about 2 ulp. e^-z overflows to infinity below z = -88; the quotient is
// then an exact 0.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

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
      const float cdf = 0.5f * erfcf(z * -0.70710678118654752f);
      a = z * cdf;
      if (GRAD) da = fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), cdf);
      break;
    }
    case Act::Sigmoid: {
      const float s = sigmoid_f(z);
      a = s;
      if (GRAD) da = s * (1.f - s);
      break;
    }
    case Act::Silu: {
      const float s = sigmoid_f(z);
      a = z * s;
      if (GRAD) da = s * fmaf(z, 1.f - s, 1.f);
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
    RAPT_ACT_CASE(Gelu)
    RAPT_ACT_CASE(Relu)
    RAPT_ACT_CASE(Sigmoid)
  }
#undef RAPT_ACT_CASE
}

}  // namespace rapt
