// act.hpp -- the activations that products end with, in fp32.
//
// All but erf's are x * sigmoid(t) = x / (1 + exp(-t)):
//   silu(x)       t = x
//   gelu_tanh(x)  t = 2 sqrt(2/pi) (x + 0.044715 x^3), since 0.5 (1 + tanh(t/2)) = sigmoid(t):
//                 no cancellation where tanh is next to -1
//   gelu(x)       0.5 x erfc(-x / sqrt 2), for the same reason not 1 + erf
#pragma once

#include <hip/hip_runtime.h>

#include "internal.hpp"

namespace fp8w {

// g / (1 + exp(-t)) * u within a few units of the last place of fp32, and zero
// where 1 + exp(-t) is above 2^126 (t below -87.3): the hardware reciprocal gives
// no subnormal numbers, and what is lost is below 88 * 2^-126 < 2^-119 of u.
// exp(-t) as 2^s times a first-order correction for what rounding s = -t
// log2 e lost, and the hardware reciprocal (an IEEE division of every output
// cost as many instructions as a third of the products at k = 2048).  A gate of
// -inf gives -inf * 0, NaN.
__device__ __forceinline__ float sigmoid_times(float g, float t, float u) {
  constexpr float kLog2E = 0x1.715476p+0f, kLog2ELow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  // Beyond 200 either way 2^s is infinite and the result zero, or it is zero
  // and the result is g * u, up to infinity.
  const float a = -__builtin_amdgcn_fmed3f(t, -200.0f, 200.0f);
  const float s = a * kLog2E;
  const float lost = __builtin_fmaf(a, kLog2ELow, __builtin_fmaf(a, kLog2E, -s));
  const float e = __builtin_amdgcn_exp2f(s) * __builtin_fmaf(lost, kLn2, 1.0f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

__device__ __forceinline__ float silu_times(float g, float u) { return sigmoid_times(g, g, u); }

__device__ __forceinline__ float gelu_tanh_times(float g, float u) {
  constexpr float kTwoRoot = 1.5957691216057308f;   // 2 sqrt(2 / pi)
  return sigmoid_times(g, kTwoRoot * __builtin_fmaf(0.044715f * g * g, g, g), u);
}

__device__ __forceinline__ float gelu(float v) { return 0.5f * v * erfcf(-0.70710678118654752f * v); }

// One value's activation (but erf's), or a gate times its value.  `act` is the
// call's.
__device__ __forceinline__ float activated(int act, float v) {
  switch (act) {
    case kActSilu: return silu_times(v, 1.0f);
    case kActGeluTanh: return gelu_tanh_times(v, 1.0f);
    case kActRelu: return v > 0.0f || v != v ? v : 0.0f;   // NaN stays
    default: return v;
  }
}
__device__ __forceinline__ float gated(int act, float g, float u) {
  return act == kActGeglu ? gelu_tanh_times(g, u) : silu_times(g, u);
}

}  // namespace fp8w
