// The activations of the fused epilogue and of its gradient, in fp32.  With
// p(t) = 1 / (1 + exp(-q(t))):
//   silu(t) = t p(t),  q = t
//   gelu(t) = t p(t),  q = 2 sqrt(2 / pi) (t + 0.044715 t^3)   (the tanh form:
//             (1 + tanh(u)) / 2 = 1 / (1 + exp(-2u)))
//   slope   = p + t p (1 - p) q'(t)
// exp is the hardware's exp2 of q log2(e), the quotient its reciprocal: each
// within about 1 ulp, so p is within 2^-24 ((1 - p) (|q| + 2) + 2) of exact,
// far below the bf16 or fp8 rounding that follows.  Every instruction counts:
// one more per output value is 1.7 us at 8192 x 6912 outputs.  exp(-q) = inf gives p = 0 and exp(-q) = 0
// gives p = 1, so large |t| needs no branch.
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

// Value and slope.  t is clamped to +-L, where p is exactly 0 or 1, so that its
// cube stays finite (the clamps keep a NaN); a clamped value needs only the
// lower one.
template <int ACT> __device__ __forceinline__ void act_value_slope(float t, float& value, float& slope) {
  if constexpr (ACT == kActNone) {
    value = t;
    slope = 1.0f;
  } else if constexpr (ACT == kActRelu) {
    value = relu(t);
    slope = t > 0.0f ? 1.0f : 0.0f;
  } else {
    constexpr float L = ACT == kActGelu ? 12.0f : 128.0f;
    const float lo = __builtin_elementwise_maximum(t, -L), tc = __builtin_elementwise_minimum(lo, L);
    constexpr float a = -kLog2e * kGelu2c, b = -kLog2e * kGelu2c * kGeluA;
    const float u = tc * tc;
    const float w = ACT == kActGelu ? tc * fmaf(u, b, a) : -kLog2e * tc;
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(w));
    const float tq = ACT == kActGelu ? tc * fmaf(u, 3.0f * kGelu2c * kGeluA, kGelu2c) : tc;  // t q'(t)
    value = lo * p;
    slope = fmaf(p * (1.0f - p), tq, p);
  }
}

}  // namespace fp8mi
