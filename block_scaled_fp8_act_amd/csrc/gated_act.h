// Activations of the gated projections, in fp32: a = act(g) and its derivative.  act is
// within 2^-20 of its value (each reciprocal and exponential off by a last place), act'
// within 2^-20 of the magnitudes that it is summed from.
#pragma once

#include "fp8blk_launch.h"

namespace fp8blk {

// e^(x + lo), |lo| far below |x|: the exponential of x's rounded product with log2 e,
// times one plus what the rounding left out, rest = x + lo - y ln 2 (ln 2 in two parts).
// y's rounding alone would cost |x| units of 2^-24.  Where 2^y is 0 or infinite the
// rest can be of any size, or NaN: the bounds make a number of it.
__device__ __forceinline__ float exp_of(float x, float lo) {
  const float y = x * 0x1.715476p+0f;                                     // log2 e
  float rest = __builtin_fmaf(y, -0x1.62e430p-1f, x);
  rest = __builtin_fmaf(y, 0x1.05c610p-29f, rest) + lo;
  return __builtin_amdgcn_exp2f(y) * (1.0f + __builtin_amdgcn_fmed3f(rest, -0.5f, 0.5f));
}

// 1 / (1 + e^-(z + lo)).  e^-z overflows to infinity below z = -88, whose reciprocal is
// 0, as it should be.
__device__ __forceinline__ float logistic(float z, float lo = 0.0f) {
  return __builtin_amdgcn_rcpf(1.0f + exp_of(-z, -lo));
}
// It, and 1 less it with digits of its own: e^-z times it, 1 where e^-z is infinite (0 times
// that is NaN, of which the minimum makes 1).
__device__ __forceinline__ float logistic_both(float z, float lo, float &rest) {
  const float e = exp_of(-z, -lo), s = __builtin_amdgcn_rcpf(1.0f + e);
  rest = __builtin_fminf(e * s, 1.0f);
  return s;
}

// The normal distribution's function and e^(-g^2 / 2), of g^2 in two parts.  Left of 0,
// with x = -g / sqrt(2) and t = 1 / (1 + x / 2), it is e^(-x^2) t Q(t): Q a polynomial
// fitted to erfc(x) e^(x^2) / (2 t) over 0 <= x <= 11 (Chebyshev points, the largest
// relative error levelled: 1.23 units of 2^-24), so that small values keep their digits;
// right of 0 one less that.  With the library's erfc, whose branches a wave takes
// together, a forward call at 515 x 1000 -> 2731 took 2 us more; correcting the
// exponential costs it 0.2 of 20.6 us.
__device__ __forceinline__ float normal(float g, float &bell) {
  const float q = g * g;
  bell = exp_of(-0.5f * q, -0.5f * __builtin_fmaf(g, g, -q));   // (0 where g^2 overflows)
  const float t =
      __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(g), 0.35355339059327376f, 1.0f));
  constexpr float q9[9] = {0.14104251563549042f,   0.14119990170001984f, 0.12146279960870743f,
                           0.10169582813978195f,   -0.014145233668386936f, 0.14024096727371216f,
                           -0.2446543574333191f,   0.14279620349407196f, -0.029638642445206642f};
  float v = q9[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) v = __builtin_fmaf(v, t, q9[i]);
  const float tail = bell * (t * v);
  return g < 0.0f ? tail : 1.0f - tail;
}

// z of the form by tanh, g (1 + tanh(z / 2)) / 2 = g / (1 + e^-z): sqrt(8 / pi) (g +
// 0.044715 g^3).  Past |g| = 12 its logistic is 1 or 0 in fp32, and a cube could overflow.
// NaN stays NaN (fmax and fmin would make a number of it, and the slope 0).
__device__ __forceinline__ float within12(float g) {
  return __builtin_elementwise_minimum(__builtin_elementwise_maximum(g, -12.0f), 12.0f);
}
// z = c (A + B c^2), A = sqrt(8 / pi), B = 0.044715 A, and what its roundings leave out:
// z passes 100, and in one part its error would be that many units of 2^-24 in the tail.
__device__ __forceinline__ float tanh_z(float c, float &lo) {
  constexpr double kA = 1.5957691216057308, kB = 0.044715 * kA;
  constexpr float a = (float)kA, b = (float)kB, al = (float)(kA - a), bl = (float)(kB - b);
  const float q = c * c, ql = __builtin_fmaf(c, c, -q);
  const float h = __builtin_fmaf(b, q, a);
  const float hl = (__builtin_fmaf(b, q, -h) + a) +
                   __builtin_fmaf(b, ql, __builtin_fmaf(bl, q, al));
  const float z = c * h;
  lo = __builtin_fmaf(c, hl, __builtin_fmaf(c, h, -z));
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == kSilu) {
    return g * logistic(g);
  } else if constexpr (ACT == kGelu) {
    float bell;
    return g * normal(g, bell);
  } else {
    float lo;
    const float z = tanh_z(within12(g), lo);
    return g * logistic(z, lo);
  }
}

// act(g) and act'(g) at once.
template <int ACT>
__device__ __forceinline__ void act_both(float g, float &a, float &slope) {
  if constexpr (ACT == kSilu) {
    float rest;
    const float s = logistic_both(g, 0.0f, rest);
    a = g * s;
    slope = s * __builtin_fmaf(g, rest, 1.0f);
  } else if constexpr (ACT == kGelu) {
    float bell;
    const float p = normal(g, bell);
    a = g * p;
    slope = __builtin_fmaf(g, 0.39894228040143268f * bell, p);
  } else {
    float lo, rest;
    const float c = within12(g), z = tanh_z(c, lo), s = logistic_both(z, lo, rest);
    const float dz = 1.59576912160573071f * __builtin_fmaf(0.134145f * c, c, 1.0f);
    a = g * s;
    slope = s * __builtin_fmaf(c * dz, rest, 1.0f);
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
