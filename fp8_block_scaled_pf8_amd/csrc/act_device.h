// Activations and their derivatives in FP32 (gfx950 / CDNA4 only); formulas in include/pf8_layer.h.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/pf8_layer.h"
#include "pf8_layer_launch.h"
#include "row_device.h"

namespace pf8 {

// 1 / (1 + exp(-x)) from the exponential and reciprocal instructions, each within a step of FP32; the product by
// log2 e adds |x| 2^-24. 0 and 1 far out: the exponential overflows to infinity or vanishes.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504088896341f));
}

// tanh(u) = 2 sigmoid(2 u) - 1, so that z (1 + tanh(u)) / 2 = z s with s = sigmoid(2 u): no difference of near values for
// z far below zero. u is a polynomial of z, taken at -20 or 20 beyond that, where the sigmoid is 0 or 1 anyway
// and the cube would overflow.
constexpr float kTanhScale = 0.79788456080286535588f, kTanhCube = 0.044715f;
__device__ __forceinline__ float tanh_sigmoid(float& z, float& z2) {
  const float near = __builtin_amdgcn_fmed3f(z, -20.0f, 20.0f);
  z = z == z ? near : z;  // the median would drop NaN (and comparisons with both ends came out as branches)
  z2 = z * z;
  constexpr float c1 = static_cast<float>(-2.0 * 1.44269504088896341 * 0.79788456080286535588);
  constexpr float c3 = static_cast<float>(-2.0 * 1.44269504088896341 * 0.79788456080286535588 * 0.044715);
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * __builtin_fmaf(c3, z2, c1)));
}

// The normal distribution Phi(z) = (1 + erf(z / sqrt 2)) / 2, and e = exp(-z^2 / 2). Below zero Phi = e h(|z|) with
// h(a) = exp(a^2 / 2) Phi(-a), a smooth function that falls as 1 / a: h(a) = t P(t), t = 1 / (1 + 0.3 a), with P of
// degree 7 fitted for the least relative error on 0 .. 14 (1.5e-7, in FP32 5e-7; beyond, e vanishes). No difference of
// near values below zero, one minus that above. Below zero the roundings of e's argument count, too: together 5e-7 + 2^-24 z^2
// of Phi, 3e-6 at -6 and 1e-5 at -13. 16 instructions with two slow ones; erff takes some 50.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170368f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, __builtin_fabsf(z), 1.0f));
  float p = 0.035674771606f;
  p = __builtin_fmaf(p, t, -0.157203072659f);
  p = __builtin_fmaf(p, t, 0.206353490033f);
  p = __builtin_fmaf(p, t, -0.053683630295f);
  p = __builtin_fmaf(p, t, 0.128561619854f);
  p = __builtin_fmaf(p, t, 0.099913493968f);
  p = __builtin_fmaf(p, t, 0.120753955764f);
  p = __builtin_fmaf(p, t, 0.119629298845f);
  const float q = e * t * p;
  return z > 0.0f ? 1.0f - q : q;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == PF8_ACT_RELU) return z <= 0.0f ? 0.0f : z;  // NaN stays NaN
  if constexpr (ACT == PF8_ACT_RELU2) return z <= 0.0f ? 0.0f : z * z;
  if constexpr (ACT == PF8_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == PF8_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if constexpr (ACT == PF8_ACT_GELU_TANH) {
    float y = z, y2;
    return z * tanh_sigmoid(y, y2);
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
    float e;
    const float p = normal_cdf(z, e);
    value = z * p;
    slope = __builtin_fmaf(z * 0.39894228040143267794f, e, p);
  } else if constexpr (ACT == PF8_ACT_GELU_TANH) {
    float y = z, y2;
    const float s = tanh_sigmoid(y, y2);
    value = z * s;
    slope = __builtin_fmaf(y * (s * (1.0f - s)), __builtin_fmaf(6.0f * kTanhScale * kTanhCube, y2, 2.0f * kTanhScale), s);
  } else {
    value = z;
    slope = 1.0f;
  }
}

// Element j of a product's bias.
__device__ __forceinline__ float bias_at(const FpropActArgs& p, int64_t j) {
  return p.bias_f32 ? static_cast<const float*>(p.bias)[j] : bf_lo(static_cast<const uint16_t*>(p.bias)[j]);
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
