// Activations of the block operators and their derivatives, in fp32.
#pragma once

#include <type_traits>

#include "tpoverlap.h"

namespace tpo {

constexpr float kGeluC = 0.79788456080286535588f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + exp(-z)).  The fast exponential's documented error is 2 + 1.2 |z|
// units in the last place and the division's 2: ten units of 2^-23 for |z| up to
// 5, and about 110 where the result is tiny (z towards -88), relative error
// 1.3e-5, a three-hundredth of the bf16 outputs' 2^-8.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// The tanh form of GELU as z sigmoid(2 c z (1 + a z^2)), since (1 + tanh v) / 2
// = sigmoid(2 v).  z^2 is held at 400, where the sigmoid is 0 or 1 to every
// bit, so that a large z gives no infinity to multiply a zero with.
__device__ __forceinline__ float gelu_sq(float z) { return fminf(z * z, 400.0f); }
__device__ __forceinline__ float gelu_sigmoid(float z, float q) {
  return sigmoid_f(2.0f * kGeluC * z * (1.0f + kGeluA * q));
}

// act(z) for a compile-time activation.  RELU keeps NaN (a comparison, not a maximum).
template <int ACT>
__device__ __forceinline__ float act_f(float z) {
  if constexpr (ACT == TPO_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == TPO_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752440f));
  if constexpr (ACT == TPO_ACT_GELU_TANH) return z * gelu_sigmoid(z, gelu_sq(z));
  if constexpr (ACT == TPO_ACT_SILU) return z * sigmoid_f(z);
  return z;
}

// act'(z).
template <int ACT>
__device__ __forceinline__ float act_grad_f(float z) {
  if constexpr (ACT == TPO_ACT_RELU) return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
  if constexpr (ACT == TPO_ACT_GELU)
    return 0.5f * (1.0f + erff(z * 0.70710678118654752440f)) + z * 0.39894228040143267794f * __expf(-0.5f * z * z);
  if constexpr (ACT == TPO_ACT_GELU_TANH) {
    const float q = gelu_sq(z), s = gelu_sigmoid(z, q);
    return s + z * (s * (1.0f - s)) * (2.0f * kGeluC) * (1.0f + 3.0f * kGeluA * q);
  }
  if constexpr (ACT == TPO_ACT_SILU) {
    const float s = sigmoid_f(z);
    return s * (1.0f + z * (1.0f - s));
  }
  return 1.0f;
}

// Calls f(integral_constant<int, act>) for a runtime activation.
template <class F>
inline cudaError_t with_act(int act, F f) {
  switch (act) {
    case TPO_ACT_RELU: return f(std::integral_constant<int, TPO_ACT_RELU>());
    case TPO_ACT_GELU: return f(std::integral_constant<int, TPO_ACT_GELU>());
    case TPO_ACT_GELU_TANH: return f(std::integral_constant<int, TPO_ACT_GELU_TANH>());
    case TPO_ACT_SILU: return f(std::integral_constant<int, TPO_ACT_SILU>());
    default: return f(std::integral_constant<int, TPO_ACT_NONE>());
  }
}

}  // namespace tpo
