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
__device__ __forceinline__ float decay_scale(float l, float a) {
  const float w = 2.0f * l;
  float q = 1.0f / 720.0f;
  q = fmaf(q, w, 1.0f / 120.0f);
  q = fmaf(q, w, 1.0f / 24.0f);
  q = fmaf(q, w, 1.0f / 6.0f);
  q = fmaf(q, w, 0.5f);
  q = fmaf(q, w, 1.0f);
  const float v = w > -0.25f ? -w * q : fmaf(-a, a, 1.0f);
  return sqrt_hw(v);
}
struct Decay {
  float a, s;
};
__device__ __forceinline__ Decay decay_f(float l) {
  const float a = exp2_hw(l * kLog2e);
  return Decay{a, decay_scale(l, a)};
}

// ------------------------------------------------------------------ pieces of the recurrence
//
// A piece of consecutive steps maps the state before it to the state after it as h -> P h + H.
// P is the product of the piece's decays and H its end state from zero.  P = 0 means exactly that
// a sequence starts inside the piece, so that nothing before it may pass, not even an infinity or
// a NaN; a product that is only too small for float32 is held at the smallest normal number
// instead (an error below 2^-126 of the state), so that a NaN before it is not lost.
constexpr float kTinyDecay = 1.17549435e-38f;
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

// V consecutive elements per lane as one load or store.
template <class IO, int V>
struct Lanes;
template <>
struct Lanes<BF16, 1> {
  using raw = uint16_t;
  static __device__ __forceinline__ float get(raw r, int) { return BF16::widen(r); }
  static __device__ __forceinline__ raw put(const float* f) { return BF16::from_float(f[0]); }
};
template <>
struct Lanes<BF16, 2> {
  using raw = uint32_t;
  static __device__ __forceinline__ float get(raw r, int v) {
    return __uint_as_float(v ? r & 0xffff0000u : r << 16);
  }
  static __device__ __forceinline__ raw put(const float* f) {
    return BF16::from_float(f[0]) | static_cast<uint32_t>(BF16::from_float(f[1])) << 16;
  }
};
template <>
struct Lanes<BF16, 4> {
  using raw = uint2;
  static __device__ __forceinline__ float get(raw r, int v) {
    return Lanes<BF16, 2>::get(v < 2 ? r.x : r.y, v & 1);
  }
  static __device__ __forceinline__ raw put(const float* f) {
    return uint2{Lanes<BF16, 2>::put(f), Lanes<BF16, 2>::put(f + 2)};
  }
};
template <>
struct Lanes<BF16, 8> {
  using raw = uint4;
  static __device__ __forceinline__ float get(raw r, int v) {
    return Lanes<BF16, 2>::get(v < 2 ? r.x : v < 4 ? r.y : v < 6 ? r.z : r.w, v & 1);
  }
  static __device__ __forceinline__ raw put(const float* f) {
    return uint4{Lanes<BF16, 2>::put(f), Lanes<BF16, 2>::put(f + 2), Lanes<BF16, 2>::put(f + 4),
                 Lanes<BF16, 2>::put(f + 6)};
  }
};
template <>
struct Lanes<F32, 1> {
  using raw = float;
  static __device__ __forceinline__ float get(raw r, int) { return r; }
  static __device__ __forceinline__ raw put(const float* f) { return f[0]; }
};
template <>
struct Lanes<F32, 2> {
  using raw = float2;
  static __device__ __forceinline__ float get(raw r, int v) { return v ? r.y : r.x; }
  static __device__ __forceinline__ raw put(const float* f) { return float2{f[0], f[1]}; }
};
template <>
struct Lanes<F32, 4> {
  using raw = float4;
  static __device__ __forceinline__ float get(raw r, int v) {
    return v == 0 ? r.x : v == 1 ? r.y : v == 2 ? r.z : r.w;
  }
  static __device__ __forceinline__ raw put(const float* f) {
    return float4{f[0], f[1], f[2], f[3]};
  }
};

// A run of consecutive rows of one array, V channels per lane: a buffer resource over exactly
// those rows, so that rows past the end read as 0 and are not written, lanes past the last channel
// pass kOffNone and do neither, and an access costs one 32-bit offset register that all arrays
// share.  The whole offset is in that register: the range check subtracts a scalar offset from
// the size, which is no check where the difference would be negative.
template <class IO, int V>
struct Rows {
  using raw = typename Lanes<IO, V>::raw;
  rsrc_t r;
  __device__ __forceinline__ raw load(uint32_t off) const {
    if constexpr (sizeof(raw) == 2)
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
    else if constexpr (sizeof(raw) == 4)
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    else if constexpr (sizeof(raw) == 8)
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    else
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  }
  __device__ __forceinline__ void store(const float* f, uint32_t off) const {
    const raw v = Lanes<IO, V>::put(f);
    using v2u = __attribute__((ext_vector_type(2))) unsigned int;
    using v4u = __attribute__((ext_vector_type(4))) unsigned int;
    if constexpr (sizeof(raw) == 2)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), r, off, 0, 0);
    else if constexpr (sizeof(raw) == 4)
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, off, 0, 0);
    else if constexpr (sizeof(raw) == 8)
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u, v), r, off, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), r, off, 0, 0);
  }
};
// `first`: the first row's element offset in the array, `bytes`: of the whole run (below 2^31).
template <class IO, int V>
__device__ __forceinline__ Rows<IO, V> rows_of(const void* base, int64_t first, uint32_t bytes) {
  return Rows<IO, V>{make_buf(static_cast<const typename IO::elem*>(base) + first, bytes)};
}

}  // namespace ss
