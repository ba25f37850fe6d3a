// activation.hpp -- the activations of the gated feed-forward block and
// their derivatives, in fp32.  The three smooth ones are v times a value s(v)
// between 0 and 1, s = 1 / (1 + e^-t) with t = v (silu) or twice the tanh
// form's argument (0.5 (1 + tanh t/2) = 1 / (1 + e^-t)), or the normal
// distribution's (gelu, normal_of): no difference of nearly equal numbers where v is far
// below zero.  The hardware's
// exponential and reciprocal (one unit in the last place each) on t log2(e)
// rounded: off by about (1 + |t|) 2^-23 of s, a fortieth of fp16's rounding at
// |t| = 100.  They give zero for results below 2^-126: s is 0 for t below -87.
#pragma once
#include "sl_ops.hpp"

namespace sl {

constexpr float kLog2e = 1.44269504088896f;
constexpr float kGeluTwoC = 1.59576912160573f;     // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kInvSqrtTwoPi = 0.398942280401433f;

__device__ __forceinline__ float sigmoid_of(float t) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * t));
}

// s = erfc(-v / sqrt 2) / 2 and e = e^(-v^2 / 2), which its derivative needs too:
// for v below zero s = e t P(t), t = 1 / (1 + 0.35 |v|), above 1 less that.  P is
// erfc(u / sqrt 2) e^(u^2 / 2) / (2 t) fitted on 0 <= u <= 14 (e is zero beyond) by least squares
// whose weights move to the largest errors (Lawson's method): off by 0.5 2^-24 of
// itself, 5.2 2^-24 as summed in fp32.  s below zero is off by up to (7 + v^2) 2^-24 of itself (9 at
// -2, 18 at -4, 65 at -8, 127 at -12.4, before the hardware's e and t): e's argument is
// rounded, which counts v^2 / 2 times; fp16's own rounding is 8192 2^-24.  (With the library's
// erfcf dg and du of 8 experts of 300 x 1000, 2.4 M of each, took 12 us, so 10.)
__device__ __forceinline__ void normal_of(float v, float& s, float& e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, __builtin_fabsf(v), 1.f));
  e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * (v * v));
  float P = -0.0291460587f;
  P = __builtin_fmaf(P, t, 0.143972304f);
  P = __builtin_fmaf(P, t, -0.255715463f);
  P = __builtin_fmaf(P, t, 0.159175482f);
  P = __builtin_fmaf(P, t, -0.023110698f);
  P = __builtin_fmaf(P, t, 0.105508346f);
  P = __builtin_fmaf(P, t, 0.119832788f);
  P = __builtin_fmaf(P, t, 0.13986188f);
  P = __builtin_fmaf(P, t, 0.139621404f);
  const float q = P * t * e;
  s = v < 0.f ? q : 1.f - q;
}

// act(v)
__device__ __forceinline__ float activate(int32_t act, float v) {
  switch (act) {
    case ACT_SILU: return v * sigmoid_of(v);
    case ACT_GELU: {
      float s, e;
      normal_of(v, s, e);
      return v * s;
    }
    case ACT_GELU_TANH: return v * sigmoid_of(kGeluTwoC * v * __builtin_fmaf(kGeluCubic * v, v, 1.f));
    default: return v < 0.f ? 0.f : v;  // a NaN stays one
  }
}

// act(v) and act'(v)
__device__ __forceinline__ void activate_with_slope(int32_t act, float v, float& a, float& slope) {
  switch (act) {
    case ACT_SILU: {
      const float s = sigmoid_of(v);
      a = v * s;
      slope = s * __builtin_fmaf(v, 1.f - s, 1.f);
      return;
    }
    case ACT_GELU: {
      float s, e;
      normal_of(v, s, e);
      a = v * s;
      slope = __builtin_fmaf(v, kInvSqrtTwoPi * e, s);
      return;
    }
    case ACT_GELU_TANH: {
      // (bounded: from 8.7e19 on v^2 leaves fp32, and infinity times the s (1 - s) = 0 that
      // |v| above 10 has is no number; at the bound, |v| = 150, s is 0 or 1 to the last bit)
      const float q = __builtin_fminf(kGeluCubic * v * v, 1e3f);
      const float s = sigmoid_of(kGeluTwoC * v * (1.f + q));
      a = v * s;
      slope = __builtin_fmaf(v * s * (1.f - s), kGeluTwoC * __builtin_fmaf(3.f, q, 1.f), s);
      return;
    }
    default:
      a = v < 0.f ? 0.f : v;
      slope = v <= 0.f ? 0.f : 1.f;
  }
}

}  // namespace sl
