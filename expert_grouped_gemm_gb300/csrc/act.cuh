// act.cuh -- activations of the linear operator and their derivatives.
//
// FAST, where the result is rounded to bf16 (2^-8 of it): the hardware's approximate base-2 exponential and
// reciprocal (2^-22 and 2^-23; one instruction each, where the intrinsics add range handling that tripled
// the epilogue's instructions). Else, in the fp32 operator and where the bf16 one returns fp32, the
// full-precision functions.
#pragma once
#include "common.cuh"

namespace moe {

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^{-z}); the limits 0 and 1 come out exactly (2^128 and beyond are infinite, 1 / inf = 0)
template <bool FAST>
__device__ __forceinline__ float sigmoid_of(float z) {
  if constexpr (FAST) return rcp_approx(1.0f + ex2_approx(-kLog2e * z));
  return 1.0f / (1.0f + expf(-z));
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kRsqrt2 = 0.7071067811865476f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;  // 1 / sqrt(2 pi)

// 1 - Phi(|z|) for the bf16 operator as e^{-z^2 / 2} times a polynomial in t = 1 / (1 + c |z|) without constant
// term. Its six coefficients and c minimise the largest relative error over [0, 14] (3.9e-6, a linear program in the
// coefficients for each c): relative, because gelu's far tail is this value and is rounded relative to itself.
// g receives e^{-z^2 / 2}.
__device__ __forceinline__ float normal_tail(float z, float* g) {
  *g = ex2_approx((-0.5f * kLog2e * z) * z);
  const float t = rcp_approx(fmaf(0.3081677230f, fabsf(z), 1.0f));
  float p = fmaf(-0.0753990016f, t, 0.1891052857f);
  p = fmaf(p, t, 0.0077191753f);
  p = fmaf(p, t, 0.1364032076f);
  p = fmaf(p, t, 0.1189822102f);
  p = fmaf(p, t, 0.1231871499f);
  return p * t * *g;
}

template <bool FAST, int ACT>
__device__ __forceinline__ float act_one(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if constexpr (ACT == MOE_ACT_GELU) {
    if constexpr (!FAST) return z * (0.5f * erfcf(-z * kRsqrt2));  // 1 + erf would cancel for negative z
    // z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|)); the second term is zero past 100, where inf 0 would be NaN
    float g;
    const float h = 0.5f * z;
    return fmaf(-fminf(fabsf(z), 100.0f), normal_tail(z, &g), h + fabsf(h));
  }
  // 0.5 (1 + tanh u) = sigmoid(2 u)
  if constexpr (ACT == MOE_ACT_GELU_TANH) return z * sigmoid_of<FAST>(z * fmaf(2.0f * kGeluC * kGeluA * z, z, 2.0f * kGeluC));
  if constexpr (ACT == MOE_ACT_SILU) return z * sigmoid_of<FAST>(z);
  return z;
}

template <bool FAST, int ACT>
__device__ __forceinline__ float act_grad_one(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if constexpr (ACT == MOE_ACT_GELU) {
    if constexpr (!FAST) return fmaf(z * kRsqrt2Pi, expf(-0.5f * z * z), 0.5f * erfcf(-z * kRsqrt2));
    float g;
    const float tail = normal_tail(z, &g);
    return fmaf(z * kRsqrt2Pi, g, z < 0.0f ? tail : 1.0f - tail);
  }
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    const float s = sigmoid_of<FAST>(z * fmaf(2.0f * kGeluC * kGeluA * z, z, 2.0f * kGeluC));
    const float c = fminf(fmaxf(z, -100.0f), 100.0f);  // s (1 - s) is zero past it, where z^2 may be infinite
    return s + c * (2.0f * s * (1.0f - s)) * kGeluC * (1.0f + 3.0f * kGeluA * c * c);
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
__device__ __forceinline__ void act_fwd(int act, const float (&z)[N], float (&y)[N]) {  // y may be z
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
      if (y != z)
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
