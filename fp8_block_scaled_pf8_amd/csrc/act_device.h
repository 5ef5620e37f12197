// Activations and their derivatives in FP32 (gfx950 / CDNA4 only); formulas in include/pf8_layer.h.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/pf8_layer.h"

namespace pf8 {

// 1 / (1 + exp(-x)) from the exponential and reciprocal instructions, each within a step of FP32; the product by
// log2 e adds |x| 2^-24. 0 and 1 far out: the exponential overflows to infinity or vanishes.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504088896341f));
}

// tanh(u) = 2 sigmoid(2 u) - 1, so that z (1 + tanh(u)) / 2 = z sigmoid(2 u): no difference of near values for
// z far below zero. u is a polynomial of z, taken at -20 or 20 beyond that, where the sigmoid is 0 or 1 anyway
// and the cube would overflow.
constexpr float kTanhScale = 0.79788456080286535588f, kTanhCube = 0.044715f;
__device__ __forceinline__ float tanh_argument2(float& z) {
  z = z > 20.0f ? 20.0f : z < -20.0f ? -20.0f : z;  // NaN stays NaN, which the median instruction would drop
  return 2.0f * kTanhScale * z * __builtin_fmaf(kTanhCube * z, z, 1.0f);
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == PF8_ACT_RELU) return z <= 0.0f ? 0.0f : z;  // NaN stays NaN
  if constexpr (ACT == PF8_ACT_RELU2) return z <= 0.0f ? 0.0f : z * z;
  if constexpr (ACT == PF8_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == PF8_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752440f));
  if constexpr (ACT == PF8_ACT_GELU_TANH) {
    float y = z;
    return z * sigmoid(tanh_argument2(y));
  }
  return z;
}

// act(z) and act'(z).
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& value, float& slope) {
  if constexpr (ACT == PF8_ACT_RELU) {
    value = act_value<ACT>(z);
    slope = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == PF8_ACT_RELU2) {
    value = act_value<ACT>(z);
    slope = z > 0.0f ? 2.0f * z : 0.0f;
  } else if constexpr (ACT == PF8_ACT_SILU) {
    const float s = sigmoid(z);
    value = z * s;
    slope = s * __builtin_fmaf(z, 1.0f - s, 1.0f);
  } else if constexpr (ACT == PF8_ACT_GELU) {
    const float p = 0.5f * (1.0f + erff(z * 0.70710678118654752440f));
    const float density = 0.39894228040143267794f * __builtin_amdgcn_exp2f(z * z * -0.72134752044448170368f);
    value = z * p;
    slope = __builtin_fmaf(z, density, p);
  } else if constexpr (ACT == PF8_ACT_GELU_TANH) {
    float y = z;
    const float s = sigmoid(tanh_argument2(y));
    value = z * s;
    slope = __builtin_fmaf(y * s * (1.0f - s), 2.0f * kTanhScale * __builtin_fmaf(3.0f * kTanhCube * y, y, 1.0f), s);
  } else {
    value = z;
    slope = 1.0f;
  }
}

// Calls f with the activation as an integral constant.
template <typename F>
inline hipError_t by_activation(int act, F f) {
  switch (act) {
    case PF8_ACT_RELU: return f(std::integral_constant<int, PF8_ACT_RELU>{});
    case PF8_ACT_RELU2: return f(std::integral_constant<int, PF8_ACT_RELU2>{});
    case PF8_ACT_SILU: return f(std::integral_constant<int, PF8_ACT_SILU>{});
    case PF8_ACT_GELU: return f(std::integral_constant<int, PF8_ACT_GELU>{});
    case PF8_ACT_GELU_TANH: return f(std::integral_constant<int, PF8_ACT_GELU_TANH>{});
    default: return f(std::integral_constant<int, PF8_ACT_NONE>{});
  }
}

}  // namespace pf8
