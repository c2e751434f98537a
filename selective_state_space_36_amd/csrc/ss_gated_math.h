// ss_gated_math.h -- the gated recurrence's per-token arithmetic, shared by its kernels.
#pragma once

#include "ss_rows.h"

namespace ss {

__device__ __forceinline__ float sqrt_hw(float x) { return __builtin_amdgcn_sqrtf(x); }
__device__ __forceinline__ float rsq_hw(float x) { return __builtin_amdgcn_rsqf(x); }
__device__ __forceinline__ float sigmoid_f(float v) {
  return rcp_hw(1.0f + exp2_hw(-v * kLog2e));
}
// sigmoid(v + bias) for nb = -bias log2(e): one fused multiply-add instead of two operations.
__device__ __forceinline__ float sigmoid_biased(float v, float nb) {
  return rcp_hw(1.0f + exp2_hw(fmaf(v, -kLog2e, nb)));
}

// 1 - a^2 for the decay a = 2^y (y = A rg log2(e) <= 0); the input's scale is its root.
//
// 1 - a^2 = -expm1(w), w = 2 y ln 2.  Near w = 0 the difference 1 - a^2 cancels, so for w > -1/4
// it is the series -w (1 + w/2 + w^2/6 + w^3/24 + w^4/120 + w^5/720), whose rest is below
// w^6/5040 = 5e-8 relative there, with the powers of 2 ln 2 in its coefficients; elsewhere
// 1 - a a as one fused multiply-add, where the one-ulp error of a grows by at most
// 2 a^2 / (1 - a^2) = 7.
__device__ __forceinline__ float one_minus_square(float y, float a) {
  constexpr double k = 1.3862943611198906;  // 2 ln 2
  float q = static_cast<float>(-k * k * k * k * k * k / 720.0);
  q = fmaf(q, y, static_cast<float>(-k * k * k * k * k / 120.0));
  q = fmaf(q, y, static_cast<float>(-k * k * k * k / 24.0));
  q = fmaf(q, y, static_cast<float>(-k * k * k / 6.0));
  q = fmaf(q, y, static_cast<float>(-k * k / 2.0));
  q = fmaf(q, y, static_cast<float>(-k));
  return y > static_cast<float>(-0.25 / k) ? y * q : fmaf(-a, a, 1.0f);
}
__device__ __forceinline__ float decay_scale(float y, float a) {
  return sqrt_hw(one_minus_square(y, a));
}

// ------------------------------------------------------------------ pieces of the recurrence
//
// A piece of consecutive steps maps the state before it to the state after it as h -> P h + H.
// P is the product of the piece's decays and H its end state from zero.  P = 0 means exactly that
// a sequence starts inside the piece, so that nothing before it may pass, not even an infinity or
// a NaN; a product that is only too small for float32 is held at the smallest normal number
// instead (an error below 2^-126 of the state), so that a NaN before it is not lost.
constexpr float kTinyDecay = 1.17549435e-38f;  // 2^-126
struct Piece {
  float P, H;
};
__device__ __forceinline__ float advance(Piece p, float h) {
  return p.P == 0.0f ? p.H : fmaf(p.P, h, p.H);
}
__device__ __forceinline__ Piece then(Piece first, Piece second) {
  const float P = first.P == 0.0f || second.P == 0.0f ? 0.0f
                                                      : fmaxf(first.P * second.P, kTinyDecay);
  return Piece{P, advance(second, first.H)};
}

}  // namespace ss
