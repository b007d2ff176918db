// Activations of the gated feed-forward block and their slopes, in float32.
#pragma once

#include "qlr_internal.h"

namespace qlr {

namespace {

// act(g) = g q: q = sigmoid(v) with v = g (SiLU) or 2 c (g + 0.044715 g^3) (GELU's tanh form: (1 + tanh(z)) / 2 = sigmoid(2 z)),
// or q = Phi(g) = erfc(-g / sqrt 2) / 2 (GELU), which keeps its digits far to the left.
constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// q, and (SLOPE) d = act'(g).
template <int ACT, bool SLOPE>
__device__ __forceinline__ float act_gate(float g, float& d) {
  if constexpr (ACT == ACT_GELU) {
    const float phi = 0.5f * erfcf(g * -0.70710678118654752f);
    if constexpr (SLOPE) d = fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), phi);
    return phi;
  } else {
    const float v = ACT == ACT_SILU ? g : kGeluC * fmaf(0.044715f * g * g, g, g);
    const float e = __expf(-v), q = __builtin_amdgcn_rcpf(1.0f + e);  // (e = Inf: q = 0)
    if constexpr (SLOPE) {
      // act' = q + g q (1 - q) dv/dg; 1 - q = e q where q is near 1
      const float w = q * (q < 0.5f ? 1.0f - q : e * q);
      if constexpr (ACT == ACT_SILU) {
        d = fmaf(g, w, q);
      } else {
        // (powers of g on the small factor: g dv grows as g^3 and is infinite past 1e13, where w has long been 0)
        const float t = w * g;
        d = fmaf(kGeluC, fmaf(0.134145f * t * g, g, t), q);
      }
    }
    return q;
  }
}

template <int ACT>
__device__ __forceinline__ float act_f(float g) {
  float d;
  return g * act_gate<ACT, false>(g, d);
}

}  // namespace

}  // namespace qlr
