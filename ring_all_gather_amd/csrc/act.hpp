// Activations and their derivatives in fp32, for the epilogues and the gradient kernel.
//   relu       max(z, 0)
//   gelu       z Phi(z), Phi the normal distribution function, by its tail 1 - Phi(a) = p(t) t
//              exp(-a^2/2), t = 1 / (1 + 0.36 a): the polynomial p (degree 6) has the least largest
//              relative error on 0 <= a <= 14 (linear program over 1600 points in 64 bits), 8.5e-7,
//              1.2e-6 in fp32 arithmetic; above a = 14 the tail is less than any normal fp32 number
//   gelu_tanh  z s(2 v), v = sqrt(2/pi) (z + 0.044715 z^3): (1 + tanh v)/2 is the logistic s(2 v)
//   silu       z s(z)
// At z = -inf gelu, gelu_tanh and silu are NaN, as -inf * 0 in these formulas is, in the forward
// pass and in the backward pass alike; the derivatives take their limits, 0 at -inf and 1 at +inf.
// A NaN z gives NaN in both, relu's too, so that it shows in the gradients as it does in the
// output.
// exp is the hardware's exp2 of x log2(e) and the reciprocal the hardware's, each good to about 1
// part in 2^22.  Rounding the exponent adds 2^-24 of |x| for each operation that makes it, so
// values are good to a relative 2^-19 + 8 2^-24 |x|, x the exponent (z, z^2/2, 2 v): the far tails
// are accurate to their own size (z = -12: better than 2^-14) until they leave the range of normal
// fp32 numbers, where they are 0.  Results are rounded to bf16 (1 part in 2^8) or summed in fp32.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ringag.h"

namespace ringag {

__device__ inline float act_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ inline float act_logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + act_exp(-x));
}

// 1 - Phi(|z|), and exp(-z^2/2).
__device__ inline float act_normal_tail(float z, float* gauss) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.36f * fabsf(z));
  const float p =
      t * (0.14371239f +
           t * (0.14178240f +
                t * (0.13966253f +
                     t * (0.02670555f +
                          t * (0.18073241f + t * (-0.17960902f + t * 0.04701345f))))));
  *gauss = __builtin_amdgcn_exp2f(z * z * -0.72134752f);
  return p * *gauss;
}

template <int ACT>
__device__ inline float act_value(float z) {
  if constexpr (ACT == RAG_ACT_RELU) return z < 0.0f ? 0.0f : z;
  else if constexpr (ACT == RAG_ACT_GELU) {
    float g;
    const float tail = act_normal_tail(z, &g);
    return z * (z < 0.0f ? tail : 1.0f - tail);
  } else if constexpr (ACT == RAG_ACT_GELU_TANH)
    return z * act_logistic(1.59576912f * z * (1.0f + 0.044715f * z * z));
  else if constexpr (ACT == RAG_ACT_SILU) return z * act_logistic(z);
  else return z;
}

// act'(z); *value receives act(z).
template <int ACT>
__device__ inline float act_slope(float z, float* value) {
  if constexpr (ACT == RAG_ACT_RELU) {
    *value = z < 0.0f ? 0.0f : z;
    return z != z ? z : z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == RAG_ACT_GELU) {
    float g;
    const float tail = act_normal_tail(z, &g), c = z < 0.0f ? tail : 1.0f - tail;
    *value = z * c;
    return g == 0.0f ? c : c + z * g * 0.39894228f;   // (0 before z can be infinite)
  } else if constexpr (ACT == RAG_ACT_GELU_TANH) {
    const float z2 = z * z;
    const float s = act_logistic(1.59576912f * z * (1.0f + 0.044715f * z2));
    *value = z * s;
    // s (1 - s) underflows before z^3 grows, except where it is already 0
    const float d = s * (1.0f - s);
    return d == 0.0f ? s : s + z * d * 1.59576912f * (1.0f + 0.134145f * z2);
  } else if constexpr (ACT == RAG_ACT_SILU) {
    const float s = act_logistic(z);
    *value = z * s;
    const float d = s * (1.0f - s);
    return d == 0.0f ? s : s + z * d;
  } else {
    *value = z;
    return 1.0f;
  }
}

// Runs f with the activation as a compile-time constant (one uniform branch); PLAIN: there is none.
template <bool PLAIN = false, class F>
__device__ inline void act_switch(int act, F&& f) {
  if constexpr (PLAIN) {
    f(std::integral_constant<int, RAG_ACT_NONE>{});
    return;
  }
  switch (act) {
    case RAG_ACT_RELU: f(std::integral_constant<int, RAG_ACT_RELU>{}); break;
    case RAG_ACT_GELU: f(std::integral_constant<int, RAG_ACT_GELU>{}); break;
    case RAG_ACT_GELU_TANH: f(std::integral_constant<int, RAG_ACT_GELU_TANH>{}); break;
    case RAG_ACT_SILU: f(std::integral_constant<int, RAG_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, RAG_ACT_NONE>{}); break;
  }
}

}  // namespace ringag
