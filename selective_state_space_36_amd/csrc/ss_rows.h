// ss_rows.h -- row accesses of the recurrent block's kernels: V channels per lane, checked by the
// buffer resource's range.
#pragma once

#include "ss_device.h"

namespace ss {

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
    // (one conversion of both: rounded apart they are shifted and joined by three more instructions)
    using f2 = __attribute__((ext_vector_type(2))) float;
    using b2 = __attribute__((ext_vector_type(2))) __bf16;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{f[0], f[1]}), b2));
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
//
// PAST: the access is marked non-temporal, so that it does not keep a place in the caches.  That is
// for calls that move more than the 256 MB Infinity Cache holds (passes_cache), where nobody finds
// their rows there again.  Training steps, never / always, timed in turn with the kernels as they
// then stood: recurrence 4 x 4096 x 5120 551 / 527 us, 8 x 2048 x 1536 189 / 179, 2 x 2048 x 1536
// (63 and 113 MB) 60.4 / 65.4; norm (loads only) 16384 x 2560 227 / 206, 10000 x 2560 142 / 123,
// 16384 x 768 (151 and 201 MB) 64 / 68; convolution (its forward's loads apart, which neighbours
// share) 4 x 4096 x 5120 191 / 170.
template <class IO, int V, bool PAST = false>
struct Rows {
  using raw = typename Lanes<IO, V>::raw;
  static constexpr int kAux = PAST ? 2 : 0;  // the instruction's nt bit
  rsrc_t r;
  __device__ __forceinline__ raw load(uint32_t off) const {
    if constexpr (sizeof(raw) == 2)
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, kAux));
    else if constexpr (sizeof(raw) == 4)
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, kAux));
    else if constexpr (sizeof(raw) == 8)
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, kAux));
    else
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kAux));
  }
  __device__ __forceinline__ void store(const float* f, uint32_t off) const {
    const raw v = Lanes<IO, V>::put(f);
    using v2u = __attribute__((ext_vector_type(2))) unsigned int;
    using v4u = __attribute__((ext_vector_type(4))) unsigned int;
    if constexpr (sizeof(raw) == 2)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), r, off, 0, kAux);
    else if constexpr (sizeof(raw) == 4)
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, off, 0, kAux);
    else if constexpr (sizeof(raw) == 8)
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u, v), r, off, 0, kAux);
    else
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), r, off, 0, kAux);
  }
};
// `first`: the first row's element offset in the array, `bytes`: of the whole run (below 2^31).
template <class IO, int V, bool PAST = false>
__device__ __forceinline__ Rows<IO, V, PAST> rows_of(const void* base, int64_t first,
                                                     uint32_t bytes) {
  return Rows<IO, V, PAST>{make_buf(static_cast<const typename IO::elem*>(base) + first, bytes)};
}

// Whether a call that moves `bytes` outgrows the Infinity Cache.
inline bool passes_cache(int64_t bytes) { return bytes > (int64_t(256) << 20); }
// The same for a kernel whose workgroups take columns of rows of `row` bytes: only where the rows
// are whole cache lines, for the parts of a line that two workgroups access have to meet in a cache
// (4 x 4096 x 5121, past the caches and not: recurrence forward 248 / 214 us, training step 882 /
// 637, convolution training step 372 / 287).
inline bool passes_cache(int64_t bytes, int64_t row) {
  return passes_cache(bytes) && row % 128 == 0;
}

}  // namespace ss
