// The activations of the fused epilogue and of its gradient, in fp32.  With
// p(t) = 1 / (1 + exp(-q(t))):
//   silu(t) = t p(t),  q = t
//   gelu(t) = t p(t),  q = 2 sqrt(2 / pi) (t + 0.044715 t^3)   (the tanh form:
//             (1 + tanh(u)) / 2 = 1 / (1 + exp(-2u)))
//   slope   = p + t p (1 - p) q'(t)
// exp is the hardware's exp2 of q log2(e), the quotient its reciprocal: each
// within about 1 ulp, so p is within 2^-24 ((1 - p) (|q| + 2) + 2) of exact,
// far below the bf16 or fp8 rounding that follows.  Every instruction counts:
// one more per output value is 1.7 us at 8192 x 6912 outputs.  exp(-q) = inf
// gives p = 0 and exp(-q) = 0 gives p = 1, so large |t| needs no branch.
#pragma once
#include "fp8mi_device.h"

namespace fp8mi {

enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kGelu2c = 1.59576912160573071f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int ACT> __device__ __forceinline__ float act_p(float t) {
  // -q(t) log2(e), the constants multiplied out
  constexpr float a = -kLog2e * kGelu2c, b = -kLog2e * kGelu2c * kGeluA;
  const float w = ACT == kActGelu ? t * fmaf(t * t, b, a) : -kLog2e * t;
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(w));
}

// Keeps a NaN.
__device__ __forceinline__ float relu(float t) { return __builtin_elementwise_maximum(t, 0.0f); }

template <int ACT> __device__ __forceinline__ float act_value(float t) {
  if constexpr (ACT == kActNone) return t;
  else if constexpr (ACT == kActRelu) return relu(t);
  else return t * act_p<ACT>(t);
}

// Value and slope, the slope as p + (p - p^2) q'(t) t with the two products
// ordered so that a zero p - p^2 meets only finite factors: t^2 is clamped to
// L^2, beyond which p is exactly 0 or 1 (the clamp keeps a NaN).  An infinite t
// gives NaN, as the formula does.  (Clamping t itself costs two instructions
// more: act_grad of 8192 x 6912 with the bias gradient 87.5 us, so 85.8.)
template <int ACT> __device__ __forceinline__ void act_value_slope(float t, float& value, float& slope) {
  if constexpr (ACT == kActNone) {
    value = t;
    slope = 1.0f;
  } else if constexpr (ACT == kActRelu) {
    value = relu(t);
    slope = t > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActGelu) {
    constexpr float L = 12.0f, a = -kLog2e * kGelu2c, b = -kLog2e * kGelu2c * kGeluA;
    const float u = __builtin_elementwise_minimum(t * t, L * L);
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * fmaf(u, b, a)));
    value = t * p;
    slope = fmaf(fmaf(-p, p, p) * fmaf(u, 3.0f * kGelu2c * kGeluA, kGelu2c), t, p);
  } else {
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * t));
    value = t * p;
    slope = fmaf(fmaf(-p, p, p), t, p);
  }
}

}  // namespace fp8mi
