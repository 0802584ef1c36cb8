// activation.cuh -- the activations of the dense products in f32, the gated product and its slopes.
#pragma once

#include "common.cuh"

namespace gb300moe {

// moe_linear_act_t.
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case MOE_LINEAR_SILU:
      return __fdividef(z, 1.0f + expf(-z));
    case MOE_LINEAR_GELU_TANH: {
      // z/2 (1 + tanh u) = z / (1 + e^-2u)
      const float u = 0.7978845608028654f * fmaf(0.044715f * z * z, z, z);
      return __fdividef(z, 1.0f + expf(-2.0f * u));
    }
    case MOE_LINEAR_RELU2: {
      const float r = fmaxf(z, 0.0f);
      return z != z ? z : r * r;
    }
    default:
      return z;
  }
}

// Gated products: act(g) and act'(g); act is MOE_ACT_SILU or MOE_ACT_GELU_TANH (a constant of
// the kernel instance, as these are evaluated next to MMAs).
//   SiLU       s = 1/(1+e^-g):           act = g s,  act' = s (1 + g (1 - s))
//   GELU-tanh  v = 2 sqrt(2/pi) (g + 0.044715 g^3), s = 1/(1+e^-v) = (1 + tanh(v/2))/2:
//                                        act = g s,  act' = s + g s (1 - s) v'
// With t = e^-v: s (1 - s) = t s^2, which does not cancel where s is next to 1.
template <int kAct>
__device__ __forceinline__ float gate_value(float g) {
  if constexpr (kAct == MOE_ACT_SILU) {
    return __fdividef(g, 1.0f + __expf(-g));
  } else {
    const float v = 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
    return __fdividef(g, 1.0f + __expf(-v));
  }
}
template <int kAct>
__device__ __forceinline__ void gate_slope(float g, float& value, float& slope) {
  if constexpr (kAct == MOE_ACT_SILU) {
    // past +-80, where t would leave f32, value and slope are those of 1 or 0 to within 2e-33
    const float c = fminf(fmaxf(g, -80.0f), 80.0f);
    const float t = __expf(-c);
    const float s = __fdividef(1.0f, 1.0f + t);
    value = g * (g < -80.0f ? 0.0f : s);
    slope = fmaf(c * t * s, s, s) + (g - g);  // NaN where g has no slope
  } else {
    // the same past v = +-80; g = +-9.6 there, and 12 keeps its powers small
    const float c = fminf(fmaxf(g, -12.0f), 12.0f);
    const float g2 = c * c;
    const float v = 1.5957691216057308f * c * fmaf(0.044715f, g2, 1.0f);
    const float t = __expf(-fminf(fmaxf(v, -80.0f), 80.0f));
    const float s = __fdividef(1.0f, 1.0f + t);
    value = g * (v < -80.0f ? 0.0f : s);
    slope = fmaf(c * t * s * 1.5957691216057308f * fmaf(0.134145f, g2, 1.0f), s, s) + (g - g);
  }
}

}  // namespace gb300moe
