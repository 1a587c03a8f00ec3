// Device-side helpers of the packed-weight operators (w4_linear.hip,
// w4_grad.hip): element types, activation functions.
#pragma once

#include "awq_device.h"

namespace awq {

// Activation types of the packed-weight operators.
template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}
// One rounding, to nearest even; infinities and NaN stay what they are.
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  return (T)v;
}

// act(g): silu g / (1 + e^-g), or the tanh form of gelu,
// g/2 (1 + tanh(c (g + a g^3))) = g / (1 + e^-2c(g + a g^3)).  Both are
// g * sigmoid(y); *slope gets the derivative p + g y' p (1 - p).  With
// e = exp(-|y|) neither p nor 1 - p is formed by cancellation.
enum W4Act { kActSilu = 0, kActGelu = 1 };
template <int ACT>
__device__ __forceinline__ float act_value(float g, float* slope) {
  constexpr float kC2 = 1.5957691216057308f, kA = 0.044715f;  // 2 sqrt(2 / pi)
  const float y = ACT == kActSilu ? g : kC2 * fmaf(kA * g * g, g, g);
  const float e = expf(-fabsf(y));
  const float inv = 1.0f / (1.0f + e);
  const float big = inv, small = e * inv;  // sigmoid(|y|), sigmoid(-|y|)
  const float p = y < 0.0f ? small : big, q = y < 0.0f ? big : small;
  if (slope) {
    const float dy = ACT == kActSilu ? 1.0f : kC2 * fmaf(3.0f * kA * g, g, 1.0f);
    // p q is 0 before y' overflows: for a finite g the product's limit is 0
    const float t = p * q;
    *slope = t == 0.0f && fabsf(g) < INFINITY ? p : fmaf(g * dy, t, p);
  }
  return g * p;
}

}  // namespace awq
