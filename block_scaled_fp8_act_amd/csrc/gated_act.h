// Activations of the gated projections, in fp32: a = act(g) and its derivative.
#pragma once

#include "fp8blk_launch.h"

namespace fp8blk {

// 1 / (1 + e^-z).  e^-z overflows to infinity below z = -88, whose reciprocal is
// 0, as it should be; the argument's rounding costs |z| 2^-24 of the result.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == kSilu) return g * logistic(g);
  // g times the normal distribution's function, by erfc so that small values keep
  // their digits
  if constexpr (ACT == kGelu) return g * (0.5f * erfcf(g * -0.70710678118654752f));
  // g (1 + tanh(z / 2)) / 2 = g / (1 + e^-z), z = sqrt(8 / pi) (g + 0.044715 g^3).
  // Past |g| = 12 the logistic is 1 or 0 in fp32, and a cube could overflow.
  const float c = __builtin_fminf(__builtin_fmaxf(g, -12.0f), 12.0f);
  return g * logistic(1.59576912160573071f * c * __builtin_fmaf(0.044715f * c, c, 1.0f));
}

__device__ __forceinline__ float act_any(int act, float g) {
  return act == kSilu ? act_value<kSilu>(g)
                      : act == kGelu ? act_value<kGelu>(g) : act_value<kGeluTanh>(g);
}

template <int ACT>
__device__ __forceinline__ float act_slope(float g) {
  if constexpr (ACT == kSilu) {
    // 1 - s is the logistic of -g, with its own digits
    return logistic(g) * __builtin_fmaf(g, logistic(-g), 1.0f);
  }
  if constexpr (ACT == kGelu) {
    const float density =
        0.39894228040143268f * __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);
    // (the density is 0 where g^2 overflows)
    return __builtin_fmaf(g, density, 0.5f * erfcf(g * -0.70710678118654752f));
  }
  const float c = __builtin_fminf(__builtin_fmaxf(g, -12.0f), 12.0f);
  const float z = 1.59576912160573071f * c * __builtin_fmaf(0.044715f * c, c, 1.0f);
  const float dz = 1.59576912160573071f * __builtin_fmaf(0.134145f * c, c, 1.0f);
  return logistic(z) * __builtin_fmaf(c * dz, logistic(-z), 1.0f);
}

__device__ __forceinline__ float slope_any(int act, float g) {
  return act == kSilu ? act_slope<kSilu>(g)
                      : act == kGelu ? act_slope<kGelu>(g) : act_slope<kGeluTanh>(g);
}

}  // namespace fp8blk
