// Activations of the linear's epilogue and their slopes, in fp32.
//
// An epilogue runs them on every element of C between the product's last MFMA
// and its stores, with nothing to hide behind, so each takes one exponential
// (v_exp_f32) and at most one reciprocal (v_rcp_f32), about 1 ulp each, far
// below the 16-bit rounding that follows.
//
// Phi(-x), the normal distribution function for x >= 0, is
//   Phi(-x) = t P(t) exp(-x^2 / 2), t = 1 / (1 + p x),
// P of degree 6, its coefficients and p fitted here to erfc (scaled by
// exp(x^2)) for the smallest relative error over 0 <= x <= 14: 6e-7, 1e-6 with
// fp32's roundings for x < 2.  Further out the exponential's argument adds
// x^2 2^-24, 8e-6 at x = 12.  So gelu's negative side keeps its relative
// precision down to fp32's smallest normal numbers; 1 - Phi serves for z > 0.
#pragma once
#include "layer_device.hpp"

namespace mc2 {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

constexpr float kLog2e = 1.44269504088896340736f;

// exp(-z^2 / 2) and Phi(z)
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.265f, __builtin_fabsf(z), 1.0f));
  e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * (z * z));
  float q = __builtin_fmaf(t, -0.067787081f, 0.195273310f);
  q = __builtin_fmaf(t, q, -0.066363186f);
  q = __builtin_fmaf(t, q, 0.142493516f);
  q = __builtin_fmaf(t, q, 0.082946517f);
  q = __builtin_fmaf(t, q, 0.107836790f);
  q = __builtin_fmaf(t, q, 0.105599828f);
  q = q * t * e;
  return z > 0.0f ? 1.0f - q : q;
}
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}
constexpr float kTanhA = 1.59576912160573071176f;            // 2 sqrt(2 / pi)
constexpr float kTanhB = 1.59576912160573071176f * 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if constexpr (ACT == ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  // 0.5 (1 + tanh u) = sigmoid(2 u)
  if constexpr (ACT == ACT_GELU_TANH) return z * sigmoid(z * __builtin_fmaf(kTanhB, z * z, kTanhA));
  if constexpr (ACT == ACT_SILU) return z * sigmoid(z);
  return z;
}

// The slopes tend to 1 and 0 where a term z (1 - p) p would be inf * 0, so z is
// taken within +-1e4 there, where that term has long been 0.  An infinite z is
// no rare input: a pre-activation past fp16's range is saved as one.  (The
// clamp drops a NaN, p keeps it.)
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  const float zc = __builtin_amdgcn_fmed3f(z, -1e4f, 1e4f);
  if constexpr (ACT == ACT_GELU) {
    float e;
    const float p = normal_cdf(z, e);
    return __builtin_fmaf(zc * 0.39894228040143267794f, e, p);
  }
  if constexpr (ACT == ACT_GELU_TANH) {
    const float z2 = zc * zc, p = sigmoid(z * __builtin_fmaf(kTanhB, z2, kTanhA));
    return __builtin_fmaf(zc * p * (1.0f - p), __builtin_fmaf(3.0f * kTanhB, z2, kTanhA), p);
  }
  if constexpr (ACT == ACT_SILU) {
    const float p = sigmoid(z);
    return __builtin_fmaf(zc * p, 1.0f - p, p);
  }
  return 1.0f;
}

// Calls f with the activation as a compile-time constant.
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>()); break;
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>()); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>()); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>()); break;
    default: f(std::integral_constant<int, ACT_NONE>());
  }
}

}  // namespace mc2
