// act.cuh - the activations of the gated feed-forward block and their derivatives,
// in float.
#pragma once

#include "common.cuh"

namespace moe {

// act(z); all of them hand a NaN on.
template <int kAct>
__device__ __forceinline__ float act_f(float z) {
  if (kAct == MOE_ACT_SILU) return silu_f(z);
  if (kAct == MOE_ACT_GELU) return 0.5f * z * erfcf(-0.70710678118654752f * z);
  if (kAct == MOE_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = 1 / (1 + e^-2u); past |z| = 16 it is 0 or 1 in float
    const float c = fminf(fmaxf(z, -16.0f), 16.0f);
    return z * sigmoid_f(c * (1.5957691216057308f + 0.07135481282742977f * c * c));
  }
  return z <= 0.0f ? 0.0f : z;
}

// act(z) and act'(z).
template <int kAct>
__device__ __forceinline__ void act_both(float z, float& f, float& d) {
  if (kAct == MOE_ACT_SILU) {
    const float s = sigmoid_f(z);
    f = z * s;
    d = s * (1.0f + z * (1.0f - s));
  } else if (kAct == MOE_ACT_GELU) {
    const float c = 0.5f * erfcf(-0.70710678118654752f * z);
    f = z * c;
    d = c + z * 0.39894228040143268f * __expf(-0.5f * z * z);
  } else if (kAct == MOE_ACT_GELU_TANH) {
    const float c = fminf(fmaxf(z, -16.0f), 16.0f);
    const float s = sigmoid_f(c * (1.5957691216057308f + 0.07135481282742977f * c * c));
    f = z * s;
    d = s + c * s * (1.0f - s) * (1.5957691216057308f + 0.21406443848228931f * c * c);
    if (z != z) d = z;
  } else {
    f = z <= 0.0f ? 0.0f : z;
    d = z <= 0.0f ? 0.0f : z > 0.0f ? 1.0f : z;
  }
}

}  // namespace moe
