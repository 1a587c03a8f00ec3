// Device-side helpers of the packed-weight operators (w4_*.hip): element types,
// activation functions, zeros in two parts, codes as fp16.
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

// The block's place in a grid_of() launch.
__device__ __forceinline__ uint32_t grid_block() { return blockIdx.y * (uint32_t)kGridRow + blockIdx.x; }

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

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Differences are held in units of 2^-9 between the codes and the step, which
// takes the factor back: a nibble in bits 0-3 of a half is the fp16 subnormal
// q 2^-24 and in bits 4-7 q 2^-20, so one packed fma by (2^15, 2^11) gives
// (q - z) 2^-9 with one rounding; none for the high part of a zero.
constexpr float kCodeScale = 512.0f;
__device__ __forceinline__ uint32_t neg_zero_pair(_Float16 z) {
  const _Float16 n = (_Float16)(-0.001953125f) * z;
  const uint32_t b = __builtin_bit_cast(uint16_t, n);
  return b | (b << 16);
}

// A zero as high + low: q - high is exact in 16 bits for all 16 codes (BF16: in
// bf16's 8 bits, else in fp16's 11) and is 0 or of the other sign only where
// q - z is, so that an infinity times it is what the formula gives; low
// multiplies the tokens' sums over the group, in fp32.
//   |z| <= 17: |q - high| <= 32, so high is a multiple of 2^-6 (2^-3), the lower
//   neighbour's odd one where z is none: never a code unless z is one.
//   Beyond, no code is near: a whole number, of magnitude up to 2032 (240).
struct ZeroParts {
  float high, low;
};
template <bool BF16>
__device__ __forceinline__ ZeroParts split_zero(float z) {
  constexpr float kParts = BF16 ? 8.0f : 64.0f, kTop = BF16 ? 240.0f : 2032.0f;
  const float v = z * kParts, f = floorf(v);
  const int i = (int)f | (f != v ? 1 : 0);
  const float high = fabsf(z) <= 17.0f ? (float)i * (1.0f / kParts)
                                       : fminf(fmaxf(__builtin_rintf(z), -kTop), kTop);
  return {high, z - high};
}
// The factors of a nibble in bits 0-3 of the low half and bits 4-7 of the
// high one, as fp16 pairs.
constexpr uint32_t kNibbleFactors = 0x68007800u;

// The eight codes of a word, in column order, as (q - z) 2^-9: ten operations.
// With factors and zero 0 they all become 0.
__device__ __forceinline__ uint4 dequant_word(uint32_t w, uint32_t nz,
                                              uint32_t factors = kNibbleFactors) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = w & 0xF0F0F0F0u;
  const half2v m = __builtin_bit_cast(half2v, factors);
  const half2v z = __builtin_bit_cast(half2v, nz);
  auto pair = [&](uint32_t sel) {
    const half2v c = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(hi, lo, sel));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c, m, z));
  };
  return make_uint4(pair(0x0c040c00u), pair(0x0c050c01u), pair(0x0c060c02u), pair(0x0c070c03u));
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// Packed fp16 to packed bf16, rounded to nearest even.
__device__ __forceinline__ uint32_t half2_to_bf16x2(uint32_t v) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 r = {(__bf16)f16_lo(v), (__bf16)f16_hi(v)};
  return __builtin_bit_cast(uint32_t, r);
}
template <typename T>
__device__ __forceinline__ floatx4 mfma16(uint4 a, uint4 b, floatx4 c) {
  if constexpr (sizeof(T) == 2 && __is_same(T, _Float16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

}  // namespace awq
