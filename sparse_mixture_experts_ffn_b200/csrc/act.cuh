// act.cuh -- the activations of the linear layer and their derivatives, in fp32.
#pragma once

#include "moe_ops.h"

namespace moe {

// 2^t and 1 / d by the hardware's approximations, each off by a step or two of fp32; results too
// small for fp32's normal numbers become zero
__device__ __forceinline__ float exp2_approx(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
__device__ __forceinline__ float rcp_approx(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

// min and max that pass NaN on
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 1 / (1 + e^-z), 0 and 1 far out, without NaN from overflow.
// FAST, for results that are rounded to bf16: the exponent z log2(e) is rounded, which costs e^-z
// about |z| 2^-24 relative, far inside half a step of bf16.  Else what was lost is put back
// to first order, 2^(t + r) = 2^t (1 + r ln 2), and the result is within 6 half steps of fp32.
// (expf and a division took three times the instructions, and arithmetic, not memory, bounded
// the gated activation.)
template <bool FAST>
__device__ __forceinline__ float sigmoid_of(float z) {
  constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;  // their sum is log2(e) to 2^-50
  if (FAST) return rcp_approx(1.0f + exp2_approx(z * -kLog2e));
  const float x = fminf(fmaxf(-z, -88.0f), 88.0f);  // 1 / (1 + e^88) is zero already
  const float t = x * kLog2e;
  const float r = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -t));
  const float e = exp2_approx(t);
  return rcp_approx(1.0f + fmaf(e, r * 0.693147181f, e));
}

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;

// Phi(z), the normal distribution's integral, and e^(-z^2 / 2) with it: Phi(-|z|) = P(t) e^(-z^2 / 2) with t =
// 1 / (1 + p |z|), the form of Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26.  Their
// coefficients keep the absolute error down (1.5e-7), which far below zero is a large part of Phi (1% at
// -8), and so does 1 + erf(z / sqrt 2) in fp32 (6% at -5, all of it from -6 on).  These are minimax fits
// of the relative error over 0 <= |z| <= 14.
// FAST, for results that are rounded to bf16: within 4.5e-4 of Phi and 6.2e-7 absolute, in as many
// instructions as with their coefficients.  Else within 1.5e-7, and 7 half steps of fp32 as evaluated, the
// exponent's lost part put back as in sigmoid_of() (normcdff: 2048 outputs of 4096 rows and 128 features
// 99 us, erff 79, like this 78).
template <bool FAST>
__device__ __forceinline__ float phi_of(float z, float& gauss) {
  constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;
  float q;
  if (FAST) {
    const float t = rcp_approx(fmaf(fabsf(z), 0.35f, 1.0f));
    gauss = exp2_approx(z * z * (-0.5f * kLog2e));
    q = fmaf(t, -0.0965571106f, 0.271923155f);
    q = fmaf(t, q, 0.0230577457f);
    q = fmaf(t, q, 0.164107740f);
    q = fmaf(t, q, 0.137468100f) * t * gauss;
  } else {
    const float a = min_nan(fabsf(z), 16.0f);  // e^-128 is zero already
    const float t = rcp_approx(fmaf(a, 0.3f, 1.0f));
    const float sq = a * a, sq_low = fmaf(a, a, -sq), x = -0.5f * sq;
    const float y = x * kLog2e;
    const float r = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -y));
    const float e = exp2_approx(y);
    gauss = fmaf(e, fmaf(r, 0.693147181f, -0.5f * sq_low), e);
    q = fmaf(t, 0.0356750973f, -0.157204285f);
    q = fmaf(t, q, 0.206355348f);
    q = fmaf(t, q, -0.0536851883f);
    q = fmaf(t, q, 0.128562361f);
    q = fmaf(t, q, 0.0999132916f);
    q = fmaf(t, q, 0.120753989f);
    q = fmaf(t, q, 0.119629301f) * t * gauss;
  }
  return z < 0.0f ? q : 1.0f - q;
}

// The tanh form of GELU by 0.5 (1 + tanh u) = sigmoid(2 u).
template <int ACT, bool FAST>
__device__ __forceinline__ float act_of(float z) {
  if (ACT == MOE_ACT_RELU) return z < 0.0f ? 0.0f : z;  // passes NaN on
  if (ACT == MOE_ACT_SILU) return z * sigmoid_of<FAST>(z);
  if (ACT == MOE_ACT_GELU) {
    float g;
    return z * phi_of<FAST>(z, g);
  }
  // z^3 may overflow: the sigmoid is then 0 or 1
  if (ACT == MOE_ACT_GELU_TANH) return z * sigmoid_of<FAST>(2.0f * kGeluC * (z + kGeluK * z * z * z));
  return z;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_slope_of(float z) {
  if (ACT == MOE_ACT_RELU) return z <= 0.0f ? 0.0f : 1.0f;
  if (ACT == MOE_ACT_SILU) {
    const float p = sigmoid_of<FAST>(z);
    return p * (1.0f + z * (1.0f - p));
  }
  if (ACT == MOE_ACT_GELU) {
    float g;
    const float phi = phi_of<FAST>(z, g);
    return fmaf(z * 0.3989422804014327f, g, phi);
  }
  if (ACT == MOE_ACT_GELU_TANH) {
    // past |z| = 12 the sigmoid is 0 or 1 to the last bit; the clamp keeps z^3 finite there
    const float y = min_nan(max_nan(z, -12.0f), 12.0f);
    const float p = sigmoid_of<FAST>(2.0f * kGeluC * (y + kGeluK * y * y * y));
    return p + 2.0f * y * p * (1.0f - p) * kGeluC * (1.0f + 3.0f * kGeluK * y * y);
  }
  return 1.0f;
}

// in place on N values, the choice made once: inside an unrolled loop, the code of all five for
// every value overruns the instruction cache
template <int N, bool FAST, int ACT>
__device__ __forceinline__ void act_each(float* z) {
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = act_of<ACT, FAST>(z[i]);
}
template <int N, bool FAST>
__device__ __forceinline__ void act_n(float* z, int act) {
  if (act == MOE_ACT_RELU) act_each<N, FAST, MOE_ACT_RELU>(z);
  else if (act == MOE_ACT_SILU) act_each<N, FAST, MOE_ACT_SILU>(z);
  else if (act == MOE_ACT_GELU) act_each<N, FAST, MOE_ACT_GELU>(z);
  else if (act == MOE_ACT_GELU_TANH) act_each<N, FAST, MOE_ACT_GELU_TANH>(z);
}
__device__ __forceinline__ float act_f32(float z, int act) {
  act_n<1, false>(&z, act);
  return z;
}

}  // namespace moe
