// Activations of the gated projections, in fp32: a = act(g) and its derivative.
#pragma once

#include "fp8blk_launch.h"

namespace fp8blk {

// 1 / (1 + e^-z).  e^-z overflows to infinity below z = -88, whose reciprocal is
// 0, as it should be; the argument's rounding costs |z| 2^-24 of the result.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// The normal distribution's function and e^(-g^2 / 2).  Left of 0, with x = -g / sqrt(2)
// and t = 1 / (1 + x / 2), it is e^(-x^2) t Q(t): Q a polynomial fitted to
// erfc(x) e^(x^2) / (2 t) over 0 <= x <= 11 (Chebyshev points, the largest relative
// error levelled: 2^-24), so that small values keep their digits; right of 0 one less
// that.  With the library's erfc, whose branches a wave takes together, a forward call
// at 515 x 1000 -> 2731 took 22.5 us instead of 20.5.
__device__ __forceinline__ float normal(float g, float &bell) {
  bell = __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);   // (0 where g^2 overflows)
  const float t =
      __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(g), 0.35355339059327376f, 1.0f));
  constexpr float q[9] = {0.14104251563549042f,   0.14119990170001984f, 0.12146279960870743f,
                          0.10169582813978195f,   -0.014145233668386936f, 0.14024096727371216f,
                          -0.2446543574333191f,   0.14279620349407196f, -0.029638642445206642f};
  float v = q[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) v = __builtin_fmaf(v, t, q[i]);
  const float tail = bell * (t * v);
  return g < 0.0f ? tail : 1.0f - tail;
}

// z of the form by tanh, g (1 + tanh(z / 2)) / 2 = g / (1 + e^-z): sqrt(8 / pi) (g +
// 0.044715 g^3).  Past |g| = 12 its logistic is 1 or 0 in fp32, and a cube could overflow.
__device__ __forceinline__ float within12(float g) {
  return __builtin_fminf(__builtin_fmaxf(g, -12.0f), 12.0f);
}
__device__ __forceinline__ float tanh_z(float c) {
  return 1.59576912160573071f * c * __builtin_fmaf(0.044715f * c, c, 1.0f);
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == kSilu) {
    return g * logistic(g);
  } else if constexpr (ACT == kGelu) {
    float bell;
    return g * normal(g, bell);
  } else {
    return g * logistic(tanh_z(within12(g)));
  }
}

// act(g) and act'(g) at once.
template <int ACT>
__device__ __forceinline__ void act_both(float g, float &a, float &slope) {
  if constexpr (ACT == kSilu) {
    const float s = logistic(g);
    a = g * s;
    slope = s * __builtin_fmaf(g, logistic(-g), 1.0f);   // (1 - s with its own digits)
  } else if constexpr (ACT == kGelu) {
    float bell;
    const float p = normal(g, bell);
    a = g * p;
    slope = __builtin_fmaf(g, 0.39894228040143268f * bell, p);
  } else {
    const float c = within12(g), z = tanh_z(c), s = logistic(z);
    const float dz = 1.59576912160573071f * __builtin_fmaf(0.134145f * c, c, 1.0f);
    a = g * s;
    slope = s * __builtin_fmaf(c * dz, logistic(-z), 1.0f);
  }
}

__device__ __forceinline__ float act_any(int act, float g) {
  return act == kSilu ? act_value<kSilu>(g)
                      : act == kGelu ? act_value<kGelu>(g) : act_value<kGeluTanh>(g);
}

__device__ __forceinline__ void both_any(int act, float g, float &a, float &slope) {
  if (act == kSilu) act_both<kSilu>(g, a, slope);
  else if (act == kGelu) act_both<kGelu>(g, a, slope);
  else act_both<kGeluTanh>(g, a, slope);
}

}  // namespace fp8blk
