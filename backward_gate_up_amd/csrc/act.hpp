// act.hpp -- the activations of the linear layer and their derivatives, in fp32.
//
//   relu       max(z, 0)
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z (1 + tanh u) / 2 = z sigma(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
//   silu       z sigma(z)
//
// Two forms: IEEE (fp32 storage) with the device math library's exp and IEEE
// division, and fast (16-bit storage) with the hardware's base-2 exponential and
// reciprocal, each about 1 fp32 ulp. What is added to 1 is never near -1 in either,
// so small values of gelu keep their relative accuracy.
//
// Phi: with a = |z|, Phi(-a) = Q(a) exp(-a^2 / 2), Q falling from 1/2 like 1 / (a
// sqrt(2 pi)). Q(a) = t p(t), t = 1 / (1 + c a), p fitted to the scaled
// complementary error function for the smallest relative error on 0 <= a <= 14
// (past that the exponential is zero): degree 8 for IEEE, 2.8e-8 in exact
// arithmetic, 7.8e-8 with the coefficients in fp32, and 4.2e-7 evaluated in fp32
// step by step, t and its roundings with it and the exponential without (the math
// library's erfc took 12 of the 67 us of T = 1000, K = 1024, N = 2816); degree 5 for
// fast, 4.8e-6, evaluated 5.0e-6, a hundredth of fp16's half step.
// The exponential also serves the derivative's density.
#pragma once
#include "gemm_tile.hpp"
#include "swiglu_mlp.h"

namespace swiglu {

constexpr float kLog2E = 1.44269504088896341f;
constexpr float kTwoRoot2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)

template <bool IEEE>
__device__ __forceinline__ float sigma(float z) {
  if constexpr (IEEE) return 1.0f / (1.0f + expf(-z));
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -kLog2E));
}

// Phi(z), and in e the exponential exp(-z^2 / 2)
template <bool IEEE>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  float q;
  if constexpr (IEEE) {
    // (z^2's rounding would cost the exponential z^2 / 2 times as much)
    const float zz = z * z, low = fmaf(z, z, -zz);
    e = expf(-0.5f * zz);
    if (zz < 250.0f) e = fmaf(e, -0.5f * low, e);  // past it e is 0, and low may be Inf - Inf
    const float t = 1.0f / fmaf(0.26f, fabsf(z), 1.0f);
    float p = fmaf(t, 0.030232531132203266f, -0.1515050749763741f);
    p = fmaf(t, p, 0.2487548244581288f);
    p = fmaf(t, p, -0.14781373399670042f);
    p = fmaf(t, p, 0.1587754273748436f);
    p = fmaf(t, p, 0.051957775022344034f);
    p = fmaf(t, p, 0.10279047793607293f);
    p = fmaf(t, p, 0.10305072218275481f);
    p = fmaf(t, p, 0.10375703693773017f);
    q = t * p * e;
  } else {
    e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2E));
    const float t = __builtin_amdgcn_rcpf(fmaf(0.31f, fabsf(z), 1.0f));
    float p = fmaf(t, -0.07392462777505246f, 0.1804370421624881f);
    p = fmaf(t, p, 0.01575984681692457f);
    p = fmaf(t, p, 0.13342148993831715f);
    p = fmaf(t, p, 0.12044346275325532f);
    p = fmaf(t, p, 0.12386048073571983f);
    q = t * p * e;
  }
  return z < 0.0f ? q : 1.0f - q;
}

// 2 u of gelu_tanh
__device__ __forceinline__ float tanh_arg(float z) {
  return z * fmaf(z * z, kTwoRoot2OverPi * 0.044715f, kTwoRoot2OverPi);
}

template <bool IEEE, int ACT>
__device__ __forceinline__ float act_f32(float z) {
  if constexpr (ACT == SWIGLU_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays
  else if constexpr (ACT == SWIGLU_ACT_GELU) {
    float e;
    return z * normal_cdf<IEEE>(z, e);
  } else if constexpr (ACT == SWIGLU_ACT_GELU_TANH) return z * sigma<IEEE>(tanh_arg(z));
  else if constexpr (ACT == SWIGLU_ACT_SILU) return z * sigma<IEEE>(z);
  else return z;
}

// The derivative. At an infinity it is the limit, 0 or 1 and not 0 times an infinity:
// z may be one because a finite sum left the storage type's range, whose y is finite.
// The factors beside z are 0 from |z| = 104 on, so z is cut off at 1000 there; a NaN
// stays one by those factors.
template <bool IEEE, int ACT>
__device__ __forceinline__ float act_slope(float z) {
  const float cut = __builtin_amdgcn_fmed3f(z, -1000.0f, 1000.0f);
  if constexpr (ACT == SWIGLU_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  else if constexpr (ACT == SWIGLU_ACT_GELU) {
    float e;
    const float c = normal_cdf<IEEE>(z, e);
    return fmaf(cut * e, 0.39894228040143268f, c);
  } else if constexpr (ACT == SWIGLU_ACT_GELU_TANH) {
    const float s = sigma<IEEE>(tanh_arg(z));
    return fmaf(cut * s * (1.0f - s), kTwoRoot2OverPi * fmaf(cut * cut, 3.0f * 0.044715f, 1.0f), s);
  } else if constexpr (ACT == SWIGLU_ACT_SILU) {
    const float s = sigma<IEEE>(z);
    return fmaf(cut * s, 1.0f - s, s);
  } else return 1.0f;
}

// The activation by its code, the same on every lane, of four values.
template <bool IEEE, int ACT>
__device__ __forceinline__ void act4_of(f32x4_t& z) {
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = act_f32<IEEE, ACT>(z[i]);
}
template <bool IEEE>
__device__ __forceinline__ void act4(int act, f32x4_t& z) {
  if (act == SWIGLU_ACT_RELU) act4_of<IEEE, SWIGLU_ACT_RELU>(z);
  else if (act == SWIGLU_ACT_GELU) act4_of<IEEE, SWIGLU_ACT_GELU>(z);
  else if (act == SWIGLU_ACT_GELU_TANH) act4_of<IEEE, SWIGLU_ACT_GELU_TANH>(z);
  else if (act == SWIGLU_ACT_SILU) act4_of<IEEE, SWIGLU_ACT_SILU>(z);
}

}  // namespace swiglu
