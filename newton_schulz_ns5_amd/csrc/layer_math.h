// Activations of the linear product and their derivatives, in fp32.
#pragma once

#include "device_util.h"
#include "muon_mi355x.h"

namespace muon {

// 1 / (1 + exp(-t)).  exp(-t) = 2^(-t log2 e) overflows to infinity below
// t = -88, where the reciprocal gives the limit 0.
__device__ __forceinline__ float logistic(float t) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896f * t));
}

// 2 sqrt(2 / pi) (z + 0.044715 z^3): 1/2 (1 + tanh(u)) = logistic(2 u).
__device__ __forceinline__ float gelu_arg(float z) {
  return 1.59576912160573f * z * (1.f + 0.044715f * z * z);
}

// The normal distribution function of z, and its density through `pdf`, with
// one exponential for both: 1/2 erfc(x) = 1/2 P(t) exp(-x^2), x = |z| / sqrt 2,
// t = 1 / (1 + 0.3275911 x) (Abramowitz and Stegun, 7.1.26: within 1.5e-7 of
// erf, at a third of the instructions of the library's erff, which cost the
// epilogue of a 4096 x 14336 product 20 us).
__device__ __forceinline__ float normal_cdf(float z, float& pdf) {
  const float e = __builtin_amdgcn_exp2f(-0.721347520444482f * z * z);
  const float t = __builtin_amdgcn_rcpf(1.f + 0.231641888f * fabsf(z));
  float q = 1.061405429f;
  q = q * t - 1.453152027f;
  q = q * t + 1.421413741f;
  q = q * t - 0.284496736f;
  q = q * t + 0.254829592f;
  const float h = 0.5f * q * t * e;
  pdf = 0.398942280401433f * e;
  return z > 0.f ? 1.f - h : h;
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == MUON_ACT_RELU) return z <= 0.f ? 0.f : z;  // a NaN stays one
  if constexpr (ACT == MUON_ACT_RELU2) return z <= 0.f ? 0.f : z * z;
  if constexpr (ACT == MUON_ACT_SILU) return z * logistic(z);
  if constexpr (ACT == MUON_ACT_GELU) {
    float pdf;
    return z * normal_cdf(z, pdf);
  }
  if constexpr (ACT == MUON_ACT_GELU_TANH) return z * logistic(gelu_arg(z));
  return z;
}

// The smooth slopes are taken at z cut to [-30, 30], beyond which they equal
// 0 or 1 to fp32's last bit, so that no infinity meets a zero.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == MUON_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == MUON_ACT_RELU2) return z > 0.f ? 2.f * z : 0.f;
  if constexpr (ACT == MUON_ACT_SILU || ACT == MUON_ACT_GELU || ACT == MUON_ACT_GELU_TANH) {
    const float c = z < -30.f ? -30.f : (z > 30.f ? 30.f : z);
    if constexpr (ACT == MUON_ACT_SILU) {
      const float s = logistic(c);
      return s * (1.f + c * (1.f - s));
    }
    if constexpr (ACT == MUON_ACT_GELU) {
      float pdf;
      const float cdf = normal_cdf(c, pdf);
      return cdf + c * pdf;
    }
    const float s = logistic(gelu_arg(c));
    return s + c * s * (1.f - s) * 1.59576912160573f * (1.f + 0.134145f * c * c);
  }
  return 1.f;
}

// `f` called with the activation as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case MUON_ACT_RELU: f(std::integral_constant<int, MUON_ACT_RELU>{}); break;
    case MUON_ACT_RELU2: f(std::integral_constant<int, MUON_ACT_RELU2>{}); break;
    case MUON_ACT_SILU: f(std::integral_constant<int, MUON_ACT_SILU>{}); break;
    case MUON_ACT_GELU: f(std::integral_constant<int, MUON_ACT_GELU>{}); break;
    case MUON_ACT_GELU_TANH: f(std::integral_constant<int, MUON_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, MUON_ACT_NONE>{}); break;
  }
}

}  // namespace muon
