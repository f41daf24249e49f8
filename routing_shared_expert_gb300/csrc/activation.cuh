// Activations of the dense projections (moe_act) and their derivatives, in fp32.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// The tanh form uses (1 + tanh u) / 2 = sigmoid(2 u).
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? z : 0.f;
    case MOE_ACT_GELU: return 0.5f * z * (1.f + erff(z * kSqrtHalf));
    case MOE_ACT_GELU_TANH:
      return z / (1.f + __expf(-kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z)));
    case MOE_ACT_SILU: return z / (1.f + __expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_GELU:
      return 0.5f * (1.f + erff(z * kSqrtHalf)) + z * __expf(-0.5f * z * z) * kInvSqrt2Pi;
    case MOE_ACT_GELU_TANH: {
      const float g = 1.f / (1.f + __expf(-kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z)));
      return g + z * g * (1.f - g) * kTwoSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z);
    }
    case MOE_ACT_SILU: {
      const float g = 1.f / (1.f + __expf(-z));
      return g + z * g * (1.f - g);
    }
    default: return 1.f;
  }
}

}  // namespace moe
