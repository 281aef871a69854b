// Activations of the linear layer and their slopes (fp32).
//
// gelu_tanh, 0.5 z (1 + tanh u) with u = sqrt(2/pi) (z + 0.044715 z^3), is
// z sigmoid(2u), and gelu is z Phi(z) with Phi(-|z|) = erfc(|z| / sqrt 2) / 2: neither
// form subtracts nearly equal numbers for negative z. The exponentials take the
// hardware's exp2, the quotients its reciprocal (1 ulp each).
//
// Phi(-|z|) = exp(-x^2) t p(t) with x = |z| / sqrt 2, t = 1 / (1 + x / 2): p is the
// degree-8 least-squares fit of erfc(x) exp(x^2) / (2 t) at 400 Chebyshev nodes of t
// in x <= 9.5 (beyond, exp(-x^2) is 0 in fp32). Evaluated in fp32 p is within 3e-7 of
// its function, relative, over the whole range.
//
// Relative error in the tails, where a value is about exp(-a): the exponent's own
// roundings, a few 2^-24 of a, become relative errors of the result. With r = 2^-24,
// silu (a = |z|) is within (2 a + 8) r, gelu_tanh (a = |2 u|) within (7 a + 8) r, and
// gelu (a = z^2 / 2) within 4e-7 + (6 a + 8) r: 4e-6 at z = -6 and 1.7e-5 near -13 in an
// emulation. Absolute errors of values and slopes stay below 2e-6 of max(1, |z|).
#pragma once

#include "common.hpp"

namespace mao {

constexpr float kLog2e = 1.4426950408889634f;
// 2 u = z (kGelu1 + kGelu3 z^2)
constexpr float kGelu1 = 1.5957691216057308f, kGelu3 = 0.07135481282553604f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float sigmoid_hw(float x) {
  return __builtin_amdgcn_rcpf(1.f + exp2_hw(-kLog2e * x));
}

// Phi(z), and e = exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float x = 0.70710678118654752f * fabsf(z);
  const float t = __builtin_amdgcn_rcpf(1.f + 0.5f * x);
  float p = -2.900725947e-02f;
  p = p * t + 1.398535119e-01f;
  p = p * t + -2.388618639e-01f;
  p = p * t + 1.339732756e-01f;
  p = p * t + -1.008252225e-02f;
  p = p * t + 1.000860364e-01f;
  p = p * t + 1.218424207e-01f;
  p = p * t + 1.411512882e-01f;
  p = p * t + 1.410450964e-01f;
  e = exp2_hw(-kLog2e * x * x);
  const float q = e * t * p;
  return z < 0.f ? q : 1.f - q;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == MAO_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays NaN
  if constexpr (ACT == MAO_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if constexpr (ACT == MAO_ACT_GELU_TANH) return z * sigmoid_hw(z * (kGelu1 + kGelu3 * z * z));
  if constexpr (ACT == MAO_ACT_SILU) return z * sigmoid_hw(z);
  return z;
}

// Beyond |z| = 30 the gelu slopes are 0 or 1 in fp32, beyond 120 silu's is;
// the clamp keeps z^2 finite. Comparisons, so NaN passes.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == MAO_ACT_NONE) return 1.f;
  if constexpr (ACT == MAO_ACT_RELU) return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
  if constexpr (ACT == MAO_ACT_SILU) {
    z = z > 120.f ? 120.f : (z < -120.f ? -120.f : z);
    const float s = sigmoid_hw(z);
    return s * (1.f + z * (1.f - s));
  }
  z = z > 30.f ? 30.f : (z < -30.f ? -30.f : z);
  if constexpr (ACT == MAO_ACT_GELU) {
    float e;
    const float cdf = normal_cdf(z, e);
    return cdf + 0.3989422804014327f * z * e;
  }
  const float z2 = z * z;
  const float s = sigmoid_hw(z * (kGelu1 + kGelu3 * z2));
  return s + z * s * (1.f - s) * (kGelu1 + 3.f * kGelu3 * z2);
}

// v[i] <- act(v[i]); act is the same for the whole launch.
template <int N>
__device__ __forceinline__ void act_apply(int act, float (&v)[N]) {
#define MAO_ACT_CASE(A)                                        \
  case A:                                                      \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = act_value<A>(v[i]); \
    break;
  switch (act) {
    MAO_ACT_CASE(MAO_ACT_RELU)
    MAO_ACT_CASE(MAO_ACT_GELU)
    MAO_ACT_CASE(MAO_ACT_GELU_TANH)
    MAO_ACT_CASE(MAO_ACT_SILU)
    default: break;
  }
#undef MAO_ACT_CASE
}

// v[i] <- v[i] * act'(z[i])
template <int N>
__device__ __forceinline__ void act_slope_apply(int act, const float (&z)[N], float (&v)[N]) {
#define MAO_ACT_CASE(A)                                        \
  case A:                                                      \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] *= act_slope<A>(z[i]); \
    break;
  switch (act) {
    MAO_ACT_CASE(MAO_ACT_RELU)
    MAO_ACT_CASE(MAO_ACT_GELU)
    MAO_ACT_CASE(MAO_ACT_GELU_TANH)
    MAO_ACT_CASE(MAO_ACT_SILU)
    default: break;
  }
#undef MAO_ACT_CASE
}

}  // namespace mao
