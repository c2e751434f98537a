// ss_scan2_bwd.h -- step sizes, decays and sums over a wave that the kernels of the multi-head
// scan's gradients share.
#pragma once

#include "ss_device.h"

namespace ss {

// Sum over the four 16-lane rows of a wave, in each of them: an exchange of odd and even rows, then
// of halves (both operands the same value: one result holds the first of each pair twice, the other
// the second).
__device__ __forceinline__ float sum_halves(float v) {
  const uint32_t w = __float_as_uint(v);
  const auto pair = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(pair[0]) + __uint_as_float(pair[1]);
}
__device__ __forceinline__ float sum_rows(float v) {
  const uint32_t w = __float_as_uint(v);
  const auto pair = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return sum_halves(__uint_as_float(pair[0]) + __uint_as_float(pair[1]));
}
__device__ __forceinline__ float sum16(float v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  return v + row_ror<1>(v);
}
__device__ __forceinline__ float sum64(float v) { return sum_rows(sum16(v)); }

// The same of float64 values.
__device__ __forceinline__ double sum_halves(double v) {
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = static_cast<uint32_t>(w), hi = static_cast<uint32_t>(w >> 32);
  const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
  const auto h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
  return __builtin_bit_cast(double, static_cast<uint64_t>(h[0]) << 32 | l[0]) +
         __builtin_bit_cast(double, static_cast<uint64_t>(h[1]) << 32 | l[1]);
}
__device__ __forceinline__ double sum_rows(double v) {
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = static_cast<uint32_t>(w), hi = static_cast<uint32_t>(w >> 32);
  const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
  const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
  return sum_halves(__builtin_bit_cast(double, static_cast<uint64_t>(h[0]) << 32 | l[0]) +
                    __builtin_bit_cast(double, static_cast<uint64_t>(h[1]) << 32 | l[1]));
}

// Inclusive sum of the log2 decays in float64, as float32 high and low parts: differences of them
// are exponents, whose error is a relative one of the result.
struct Step {
  float dt, slope;           // the step and its derivative by dt (input + bias)
  float c_hi, c_lo;
  float before, after, end;  // 2^{c}, 2^{c_end - c}, 2^{c_end}
};
// x plus the value that the DPP control brings (0 where it brings none), in the rows of the mask.
template <int CTRL, int ROWS, bool CLEAR>
__device__ __forceinline__ double dpp_add(double x) {
  const uint64_t w = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), CTRL, ROWS, 0xf, CLEAR);
  const uint32_t hi =
      __builtin_amdgcn_update_dpp(0, static_cast<int>(w >> 32), CTRL, ROWS, 0xf, CLEAR);
  return x + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// Over the 16 lanes of a row (each has its source), in each of them.
__device__ __forceinline__ double sum16(double v) {
  v = dpp_add<0x128, 0xf, true>(v);
  v = dpp_add<0x124, 0xf, true>(v);
  v = dpp_add<0x122, 0xf, true>(v);
  return dpp_add<0x121, 0xf, true>(v);
}
// Inclusive sum over the 64 lanes, as wave_prefix_sum.
__device__ __forceinline__ double scan64(double x) {
  x = dpp_add<0x111, 0xf, true>(x);
  x = dpp_add<0x112, 0xf, true>(x);
  x = dpp_add<0x114, 0xf, true>(x);
  x = dpp_add<0x118, 0xf, true>(x);
  x = dpp_add<0x142, 0xa, false>(x);
  return dpp_add<0x143, 0xc, false>(x);
}
__device__ __forceinline__ double last_lane(double x) {
  const uint64_t w = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(w), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(w >> 32), 63);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// e^x for x <= 0, the rounding of x log2(e) made good (it would cost |x| half steps of the result:
// a hundred steps' sum of the decays' gradient showed it, 1.4e-6 against 3e-7).
__device__ __forceinline__ float exp_neg(float x) {
  x = x < -110.0f ? -110.0f : x;  // (0 below; a NaN stays one)
  const float hi = x * kLog2e, lo = fmaf(x, kLog2e, -hi) + x * 1.925963e-8f;
  return exp2_hw(hi) * fmaf(lo, kLn2, 1.0f);
}
// 2^x, x in float64: what x loses in float32, half a step of up to 1000, is put back.
__device__ __forceinline__ float exp2_of(double x) {
  const float hi = static_cast<float>(x);
  return exp2_hw(hi) * fmaf(static_cast<float>(x - hi), kLn2, 1.0f);
}
// 2^{c_t - c_s} of two such sums, c_t the one of the larger size: what the difference of the high
// parts loses is found exactly and goes with that of the low ones.
__device__ __forceinline__ float exp2_diff(float t_hi, float t_lo, float s_hi, float s_lo) {
  const float d = t_hi - s_hi, lost = (t_hi - d) - s_hi;
  return exp2_hw(d) * fmaf(lost + (t_lo - s_lo), kLn2, 1.0f);
}
__device__ __forceinline__ Step step_of(float dt, bool in, float bias, float A, bool softplus) {
  Step s;
  const float raw = dt + bias;
  s.dt = raw;
  s.slope = 1.0f;
  if (softplus) {  // max(raw, 0) + log1p(e), with what 1 + e loses of e put back
    const float e = exp_neg(-fabsf(raw)), w = 1.0f + e, r = rcp_hw(w);
    s.dt = (raw > 0.0f ? raw : 0.0f) + (log2_hw(w) * kLn2 + (e - (w - 1.0f)) * r);
    s.slope = raw >= 0.0f ? r : e * r;
  }
  s.dt = in ? s.dt : 0.0f;
  // A step's decay below 2^-10^6 is 0 with all its products.  Held there (and at 2^10^6), sums of 64
  // of them stay in float32's range, and so do their differences: an A of the type's lowest value,
  // which lets no state through, would give infinity less infinity.
  double log2a = static_cast<double>(s.dt) * A * 1.4426950408889634;
  log2a = log2a < -1e6 ? -1e6 : log2a > 1e6 ? 1e6 : log2a;
  const double c = scan64(log2a);
  const double end = last_lane(c);
  s.c_hi = static_cast<float>(c);
  s.c_lo = static_cast<float>(c - s.c_hi);
  s.before = exp2_of(c);
  s.after = exp2_of(end - c);
  s.end = exp2_of(end);
  return s;
}

}  // namespace ss
