// Activations of the dense projections (moe_act) and their derivatives, in fp32 on the fast
// exponential and reciprocal.  The exponential is off by about (2 + 1.2 |x|) 2^-23 of its result; in a
// sigmoid s the factor s (1 - s) |x| <= 0.23 holds that at a few 2^-23 of the activation's scale, far below the
// bf16 rounding of the operands.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

__device__ __forceinline__ float fast_sigmoid(float x) { return rcp_ftz(1.f + exp_ftz(-x)); }

// The normal distribution function Phi(z) and e = exp(-z^2 / 2), by the rational
// approximation 7.1.26 of Abramowitz and Stegun: erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2)
// with t = 1 / (1 + 0.3275911 x), absolute error at most 1.5e-7 (1.3 2^-23 in Phi, which is within the
// oracle's bound of 16 2^-23 (1 + |z|) for z Phi).  The negative side takes the tail itself, so nothing
// cancels there; relative to the tail the approximation is off by 5e-4 at z = -4 and 4e-3 at
// -6, where z Phi(z) is -1.3e-4 and -6e-9.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = rcp_ftz(1.f + 0.3275911f * x);
  e = exp_ftz(-x * x);
  const float half_erfc =
      0.5f * e * t *
      (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
  return z < 0.f ? half_erfc : 1.f - half_erfc;
}

// The tanh form of GELU uses (1 + tanh u) / 2 = sigmoid(2 u).
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == MOE_ACT_RELU) return z <= 0.f ? 0.f : z;   // NaN stays
  if (ACT == MOE_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if (ACT == MOE_ACT_GELU_TANH)
    return z * fast_sigmoid(kTwoSqrt2OverPi * z * (1.f + kGeluCubic * z * z));
  if (ACT == MOE_ACT_SILU) return z * fast_sigmoid(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == MOE_ACT_RELU) return z <= 0.f ? 0.f : 1.f;
  if (ACT == MOE_ACT_GELU) {
    float e;
    const float p = normal_cdf(z, e);
    return p + z * e * 0.39894228040143268f;   // z times the density
  }
  if (ACT == MOE_ACT_GELU_TANH) {
    const float g = fast_sigmoid(kTwoSqrt2OverPi * z * (1.f + kGeluCubic * z * z));
    return g + z * g * (1.f - g) * kTwoSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z);
  }
  if (ACT == MOE_ACT_SILU) {
    const float g = fast_sigmoid(z);
    return g + z * g * (1.f - g);
  }
  return 1.f;
}

// f<ACT>() for the run-time activation.
#define MOE_DISPATCH_ACT(act, CALL)                  \
  switch (act) {                                     \
    case MOE_ACT_RELU: return CALL(MOE_ACT_RELU);    \
    case MOE_ACT_GELU: return CALL(MOE_ACT_GELU);    \
    case MOE_ACT_GELU_TANH: return CALL(MOE_ACT_GELU_TANH); \
    case MOE_ACT_SILU: return CALL(MOE_ACT_SILU);    \
    default: return CALL(MOE_ACT_NONE);              \
  }

}  // namespace moe
