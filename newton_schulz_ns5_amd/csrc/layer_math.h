// Activations of the linear product and their derivatives, in fp32.
#pragma once

#include "device_util.h"
#include "muon_mi355x.h"

namespace muon {

// BF: bf16 operands, where the short forms below stay 2^-17 (relative) or
// nearer to the definition down to the tails that fp32 holds; fp32 operands
// take the library's functions, within 2^-20 of it (what they cost is lost
// beside an fp32 product: ten times a bf16 one).

// 1 / (1 + exp(-t)).  exp(-t) overflows to infinity below t = -88, where the
// reciprocal gives the limit 0.  The short form rounds -t log2 e before it is
// raised: |t| 2^-24 of the result.
template <bool BF>
__device__ __forceinline__ float logistic(float t) {
  const float e = BF ? __builtin_amdgcn_exp2f(-1.44269504088896f * t) : expf(-t);
  return __builtin_amdgcn_rcpf(1.f + e);
}

// 2 sqrt(2 / pi) (z + 0.044715 z^3): 1/2 (1 + tanh(u)) = logistic(2 u).
__device__ __forceinline__ float gelu_arg(float z) {
  return 1.59576912160573f * z * (1.f + 0.044715f * z * z);
}

// The normal distribution function of z, and its density through `pdf`.  The
// short form has one exponential for both: the function of -|z| is
// t Q(t) exp(-z^2 / 2), t = 1 / (1 + 0.21 |z|), Q of degree 8 fitted to it here
// in the largest relative error over |z| <= 14 (1.6e-8; the rest is fp32's).
// The library's erff costs the epilogue of a 4096 x 14336 bf16 product 20 us
// more.
template <bool BF>
__device__ __forceinline__ float normal_cdf(float z, float& pdf) {
  if constexpr (!BF) {
    const float s = z * z, e = expf(-0.5f * s);
    pdf = 0.398942280401433f * fmaf(-0.5f * fmaf(z, z, -s), e, e);  // with what rounding z^2 left
    return normcdff(z);
  }
  const float e = __builtin_amdgcn_exp2f(-0.721347520444482f * z * z);
  const float t = __builtin_amdgcn_rcpf(1.f + 0.21f * fabsf(z));
  float q = -0.0716562772f;
  q = q * t + 0.283588417f;
  q = q * t - 0.330253083f;
  q = q * t + 0.349400679f;
  q = q * t - 0.0939249892f;
  q = q * t + 0.12487264f;
  q = q * t + 0.0691921909f;
  q = q * t + 0.0850688552f;
  q = q * t + 0.0837115758f;
  const float h = q * t * e;
  pdf = 0.398942280401433f * e;
  return z > 0.f ? 1.f - h : h;
}

template <int ACT, bool BF>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == MUON_ACT_RELU) return z <= 0.f ? 0.f : z;  // a NaN stays one
  if constexpr (ACT == MUON_ACT_RELU2) return z <= 0.f ? 0.f : z * z;
  if constexpr (ACT == MUON_ACT_SILU) return z * logistic<BF>(z);
  if constexpr (ACT == MUON_ACT_GELU) {
    float pdf;
    return z * normal_cdf<BF>(z, pdf);
  }
  if constexpr (ACT == MUON_ACT_GELU_TANH) return z * logistic<BF>(gelu_arg(z));
  return z;
}

// The smooth slopes are taken at z cut to where they are 0 or 1 in fp32
// (silu's, z exp(z) on its left, at -100: 4e-42; the gelus' at 30), so that no
// infinity meets a zero.
template <int ACT, bool BF>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == MUON_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == MUON_ACT_RELU2) return z > 0.f ? 2.f * z : 0.f;
  if constexpr (ACT == MUON_ACT_SILU || ACT == MUON_ACT_GELU || ACT == MUON_ACT_GELU_TANH) {
    constexpr float end = ACT == MUON_ACT_SILU ? 100.f : 30.f;
    const float c = z < -end ? -end : (z > end ? end : z);
    if constexpr (ACT == MUON_ACT_SILU) {
      const float s = logistic<BF>(c);
      return s * (1.f + c * (1.f - s));
    }
    if constexpr (ACT == MUON_ACT_GELU) {
      float pdf;
      const float cdf = normal_cdf<BF>(c, pdf);
      return cdf + c * pdf;
    }
    const float s = logistic<BF>(gelu_arg(c));
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
