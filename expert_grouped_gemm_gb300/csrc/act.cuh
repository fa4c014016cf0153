// act.cuh -- activations of the linear operator and their derivatives.
//
// The bf16 operator evaluates them with the hardware exponential and the approximate divide
// (errors of a few 1e-7 next to a rounding of 2e-3); the fp32 one with the full-precision
// functions, so that its results keep fp32 accuracy.
#pragma once
#include "common.cuh"

namespace moe {

template <bool FAST>
__device__ __forceinline__ float sigmoid_of(float z) {
  if constexpr (FAST) return sigmoidf_(z);
  return 1.0f / (1.0f + expf(-z));
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kRsqrt2 = 0.7071067811865476f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;  // 1 / sqrt(2 pi)

template <bool FAST>
__device__ __forceinline__ float act_fwd(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * kRsqrt2));
    // 0.5 (1 + tanh u) = sigmoid(2 u)
    case MOE_ACT_GELU_TANH: return z * sigmoid_of<FAST>(2.0f * kGeluC * (z + kGeluA * z * z * z));
    case MOE_ACT_SILU: return z * sigmoid_of<FAST>(z);
    default: return z;
  }
}

template <bool FAST>
__device__ __forceinline__ float act_grad(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case MOE_ACT_GELU: {
      const float e = FAST ? __expf(-0.5f * z * z) : expf(-0.5f * z * z);
      return 0.5f * (1.0f + erff(z * kRsqrt2)) + z * e * kRsqrt2Pi;
    }
    case MOE_ACT_GELU_TANH: {
      const float s = sigmoid_of<FAST>(2.0f * kGeluC * (z + kGeluA * z * z * z));
      // z s (1 - s) 2 u'(z): s (1 - s) is zero where u' overflows
      return s + z * (2.0f * s * (1.0f - s)) * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
    }
    case MOE_ACT_SILU: {
      const float s = sigmoid_of<FAST>(z);
      return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
  }
}

}  // namespace moe
