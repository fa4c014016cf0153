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

// Q(x) = erfc(|x|) e^{x^2} for the error function, by formula 7.1.26 of Abramowitz and Stegun,
// Handbook of Mathematical Functions: erf(|x|) = 1 - Q e^{-x^2} with an error of at most 1.5e-7.
__device__ __forceinline__ float erfc_scaled(float ax) {
  const float t = __fdividef(1.0f, fmaf(0.3275911f, ax, 1.0f));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  return p * t;
}

// Phi(z) = (1 + erf(z / sqrt 2)) / 2 and, through g, e^{-z^2 / 2}
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float* g) {
  if constexpr (FAST) {
    *g = __expf(-0.5f * z * z);
    const float tail = 0.5f * erfc_scaled(fabsf(z) * kRsqrt2) * *g;  // 1 - Phi(|z|)
    return z < 0.0f ? tail : 1.0f - tail;
  } else {
    *g = expf(-0.5f * z * z);
    return 0.5f * (1.0f + erff(z * kRsqrt2));
  }
}

template <bool FAST, int ACT>
__device__ __forceinline__ float act_one(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if constexpr (ACT == MOE_ACT_GELU) {
    float g;
    return z * normal_cdf<FAST>(z, &g);
  }
  // 0.5 (1 + tanh u) = sigmoid(2 u)
  if constexpr (ACT == MOE_ACT_GELU_TANH) return z * sigmoid_of<FAST>(2.0f * kGeluC * (z + kGeluA * z * z * z));
  if constexpr (ACT == MOE_ACT_SILU) return z * sigmoid_of<FAST>(z);
  return z;
}

template <bool FAST, int ACT>
__device__ __forceinline__ float act_grad_one(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if constexpr (ACT == MOE_ACT_GELU) {
    float g;
    const float phi = normal_cdf<FAST>(z, &g);
    return fmaf(z * kRsqrt2Pi, g, phi);
  }
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    const float s = sigmoid_of<FAST>(2.0f * kGeluC * (z + kGeluA * z * z * z));
    return s + z * (2.0f * s * (1.0f - s)) * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
  }
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoid_of<FAST>(z);
    return s * (1.0f + z * (1.0f - s));
  }
  return 1.0f;
}

// One branch for the whole vector: the values of a vector are independent chains, which a
// branch inside the loop would run one after the other.
template <bool FAST, int N>
__device__ __forceinline__ void act_fwd(int act, const float (&z)[N], float (&y)[N]) {
  switch (act) {
#define MOE_ACT_CASE(A)                                                    \
  case A: {                                                                \
    _Pragma("unroll") for (int i = 0; i < N; ++i) y[i] = act_one<FAST, A>(z[i]); \
    break;                                                                 \
  }
    MOE_ACT_CASE(MOE_ACT_RELU)
    MOE_ACT_CASE(MOE_ACT_GELU)
    MOE_ACT_CASE(MOE_ACT_GELU_TANH)
    MOE_ACT_CASE(MOE_ACT_SILU)
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = z[i];
#undef MOE_ACT_CASE
  }
}

// d[i] *= act'(z[i])
template <bool FAST, int N>
__device__ __forceinline__ void act_grad_mul(int act, const float (&z)[N], float (&d)[N]) {
  switch (act) {
#define MOE_ACT_CASE(A)                                                          \
  case A: {                                                                      \
    _Pragma("unroll") for (int i = 0; i < N; ++i) d[i] *= act_grad_one<FAST, A>(z[i]); \
    break;                                                                       \
  }
    MOE_ACT_CASE(MOE_ACT_RELU)
    MOE_ACT_CASE(MOE_ACT_GELU)
    MOE_ACT_CASE(MOE_ACT_GELU_TANH)
    MOE_ACT_CASE(MOE_ACT_SILU)
    default: break;
#undef MOE_ACT_CASE
  }
}

}  // namespace moe
