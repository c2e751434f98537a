// ss_gated_math.h -- the gated recurrence's per-token arithmetic, shared by its kernels.
#pragma once

#include "ss_device.h"

namespace ss {

__device__ __forceinline__ float sqrt_hw(float x) { return __builtin_amdgcn_sqrtf(x); }
__device__ __forceinline__ float sigmoid_f(float v) {
  return rcp_hw(1.0f + exp2_hw(-v * kLog2e));
}

// The decay a = e^l and the input's scale s = sqrt(1 - a^2) for l = A rg <= 0.
//
// 1 - a^2 = -expm1(w), w = 2 l.  Near w = 0 the difference 1 - a^2 cancels, so for |w| < 1/4 it is
// the series -w (1 + w/2 + w^2/6 + w^3/24 + w^4/120 + w^5/720), whose rest is below w^6/5040 =
// 5e-8 relative there; elsewhere 1 - a a as one fused multiply-add, where the one-ulp error of a
// grows by at most 2 a^2 / (1 - a^2) = 7.
struct Decay {
  float a, s;
};
__device__ __forceinline__ Decay decay_f(float l) {
  const float a = exp2_hw(l * kLog2e);
  const float w = 2.0f * l;
  float q = 1.0f / 720.0f;
  q = fmaf(q, w, 1.0f / 120.0f);
  q = fmaf(q, w, 1.0f / 24.0f);
  q = fmaf(q, w, 1.0f / 6.0f);
  q = fmaf(q, w, 0.5f);
  q = fmaf(q, w, 1.0f);
  const float v = w > -0.25f ? -w * q : fmaf(-a, a, 1.0f);
  return Decay{a, sqrt_hw(v)};
}

}  // namespace ss
