// act.h -- the gated block's activations, as device functions (gated.hip, gemv.hip).
#pragma once

#include "common.h"

namespace qnf4 {

// act(z) and its derivative, in fp32.
//   silu       z q,  q = 1 / (1 + exp(-z));          derivative q + z q (1 - q)
//   gelu       z c,  c = erfc(-z / sqrt 2) / 2;      derivative c + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z q(2 t),  t = sqrt(2 / pi) (z + 0.044715 z^3)  (1/2 (1 + tanh t) = q(2 t))
// 1 - q is formed as q(-z): no cancellation where q is near 1.
// The reciprocal is the hardware's, good to one ulp: an IEEE division would be most of what a value
// costs in the epilogue of the gated GEMM.
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }
constexpr float kTanhA = 1.5957691216057308f;           // 2 sqrt(2 / pi)
constexpr float kTanhB = kTanhA * 0.044715f;
// The cubic's argument: beyond 30 q is 0 or 1, and z^3 must not leave fp32's range.
__device__ __forceinline__ float limited(float z) { return fminf(fmaxf(z, -30.f), 30.f); }
__device__ __forceinline__ float tanh_arg(float z) {
  const float l = limited(z);
  return l * fmaf(kTanhB * l, l, kTanhA);
}
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == QLORA_ACT_SILU) return z * sigmoid(z);
  else if constexpr (ACT == QLORA_ACT_GELU) return z * (0.5f * erfcf(-0.70710678118654752f * z));
  else return z * sigmoid(tanh_arg(z));
}
template <int ACT>
__device__ __forceinline__ void act_grad(float z, float& value, float& slope) {
  if constexpr (ACT == QLORA_ACT_GELU) {
    const float c = 0.5f * erfcf(-0.70710678118654752f * z);
    value = z * c;
    slope = fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), c);
  } else if constexpr (ACT == QLORA_ACT_SILU) {
    const float q = sigmoid(z);
    value = z * q;
    slope = fmaf(value, sigmoid(-z), q);
  } else {
    const float t = tanh_arg(z), q = sigmoid(t), zl = limited(z);
    value = z * q;
    slope = fmaf(value * sigmoid(-t), fmaf(3.f * kTanhB * zl, zl, kTanhA), q);
  }
}

}  // namespace qnf4
