// activation.hpp -- the activations of the gated feed-forward block and
// their derivatives, in fp32.  The three smooth ones are v times a value s(v)
// between 0 and 1, s = 1 / (1 + e^-t) with t = v (silu) or twice the tanh
// form's argument (0.5 (1 + tanh t/2) = 1 / (1 + e^-t)), or erfc (gelu): no
// difference of nearly equal numbers where v is far below zero.  The hardware's
// exponential and reciprocal (one unit in the last place each) on t log2(e)
// rounded: off by about (1 + |t|) 2^-23 of s, an eighth of fp16's rounding at
// |t| = 100.  They give zero for results below 2^-126: s is 0 for t below -87.
#pragma once
#include "sl_ops.hpp"

namespace sl {

constexpr float kLog2e = 1.44269504088896f;
constexpr float kGeluTwoC = 1.59576912160573f;     // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kSqrtHalf = 0.707106781186548f;
constexpr float kInvSqrtTwoPi = 0.398942280401433f;

__device__ __forceinline__ float sigmoid_of(float t) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * t));
}

// act(v)
__device__ __forceinline__ float activate(int32_t act, float v) {
  switch (act) {
    case ACT_SILU: return v * sigmoid_of(v);
    case ACT_GELU: return 0.5f * v * erfcf(-kSqrtHalf * v);
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
      const float s = 0.5f * erfcf(-kSqrtHalf * v);
      a = v * s;
      slope = __builtin_fmaf(v, kInvSqrtTwoPi * __builtin_amdgcn_exp2f(-0.5f * kLog2e * v * v), s);
      return;
    }
    case ACT_GELU_TANH: {
      const float q = kGeluCubic * v * v;
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
