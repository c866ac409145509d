// Activations of the gated feed-forward, f(g), and their derivatives, in fp32.
#pragma once

#include <hip/hip_runtime.h>

namespace mxq {

// Same values as mxq_activation in mxq.h.
enum : int { ACT_SILU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3 };

// 1 / (1 + e^-z); e^-z may overflow to infinity, whose reciprocal is 0.  The hardware's
// exponential and reciprocal: |z| 2**-24 of relative error at most, 5e-6 where
// e^-z is finite, against the 2**-9 of the result's rounding.  The library's
// would cost as much in a tile's epilogue as a fifth of a K = 4096 product.
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// f(g) and, with DERIV, f'(g).
template <bool DERIV>
__device__ __forceinline__ float activation(int act, float g, float* d = nullptr) {
  if (act == ACT_SILU) {   // g s, s = logistic(g); f' = s (1 + g (1 - s))
    const float s = logistic(g);
    if constexpr (DERIV) *d = s * fmaf(g, 1.f - s, 1.f);
    return g * s;
  }
  if (act == ACT_GELU) {   // g P, P = erfc(-g / sqrt 2) / 2; f' = P + g e^(-g^2 / 2) / sqrt(2 pi)
    const float p = 0.5f * erfcf(-0.70710678f * g);
    if constexpr (DERIV) *d = fmaf(0.39894228f * g, __expf(-0.5f * g * g), p);
    return g * p;
  }
  // g (1 + tanh z) / 2 = g s, s = logistic(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3);
  // f' = s + g 2 z' s (1 - s).  Past |g| = 30 s (1 - s) is 0 in fp32, and g is held
  // there so that no power of it overflows.  A NaN is held too by the minimum and maximum
  // (one instruction): f is NaN by its factor g, but f' has none, so there it passes.
  float c = fminf(fmaxf(g, -30.f), 30.f);
  if constexpr (DERIV) c = g == g ? c : g;
  const float s = logistic(1.59576912f * c * fmaf(0.044715f * c, c, 1.f));
  if constexpr (DERIV) *d = fmaf(1.59576912f * c * fmaf(0.134145f * c, c, 1.f), s * (1.f - s), s);
  return g * s;
}

}  // namespace mxq
