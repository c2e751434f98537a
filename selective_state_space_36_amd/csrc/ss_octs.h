// ss_octs.h -- rows taken eight consecutive columns a lane (an "oct"), by the RMS norm, the gated
// norm and dropout: accesses of any alignment, sums over the lanes of a row, and the layout of rows
// on lanes.
#pragma once

#include "ss_device.h"

namespace ss {

// Sixteen bytes at the alignment of one element.
template <class E>
struct OctBytes;
template <>
struct OctBytes<uint16_t> {
  typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct OctBytes<float> {
  typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4)));
};

// Eight elements on their way, as loaded.
template <class IO>
struct Oct {
  static constexpr int kWords = sizeof(typename IO::elem) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (kWords == 8) return __uint_as_float(w[j]);
    else return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
  }
};

// Eight elements at `p`, of which n are there (n >= 8: all of them, in 16-byte accesses of whatever
// alignment the row has; fewer: one by one, the rest 0; n <= 0: none).  PAST: non-temporal.
template <class IO, bool PAST = false>
__device__ __forceinline__ Oct<IO> load_oct(const typename IO::elem* p, int n) {
  using E = typename IO::elem;
  using raw = typename OctBytes<E>::raw;
  Oct<IO> o;
  if (n >= 8) {
    const raw* q = reinterpret_cast<const raw*>(p);
#pragma unroll
    for (int h = 0; h < Oct<IO>::kWords / 4; ++h) {
      const raw a = PAST ? __builtin_nontemporal_load(q + h) : q[h];
#pragma unroll
      for (int j = 0; j < 4; ++j) o.w[4 * h + j] = a[j];
    }
  } else {
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e[j] = 0;
      if (j < n) {
        if constexpr (sizeof(E) == 4) e[j] = __float_as_uint(p[j]);
        else e[j] = p[j];
      }
    }
#pragma unroll
    for (int j = 0; j < Oct<IO>::kWords; ++j)
      o.w[j] = sizeof(E) == 4 ? e[j] : e[(2 * j) & 7] | e[(2 * j + 1) & 7] << 16;
  }
  return o;
}
template <class IO>
__device__ __forceinline__ void load8(const typename IO::elem* p, int n, float (&v)[8]) {
  const Oct<IO> o = load_oct<IO>(p, n);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = o[j];
}

template <class IO>
__device__ __forceinline__ void store8(typename IO::elem* p, int n, const float (&v)[8]) {
  using E = typename IO::elem;
  using raw = typename OctBytes<E>::raw;
  if (n >= 8) {
    raw* q = reinterpret_cast<raw*>(p);
    if constexpr (sizeof(E) == 2) {
      using f2 = __attribute__((ext_vector_type(2))) float;
      using b2 = __attribute__((ext_vector_type(2))) __bf16;
      raw a;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[j] = __builtin_bit_cast(uint32_t,
                                  __builtin_convertvector((f2{v[2 * j], v[2 * j + 1]}), b2));
      *q = a;
    } else {
      raw a, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = __float_as_uint(v[j]);
        b[j] = __float_as_uint(v[4 + j]);
      }
      q[0] = a;
      q[1] = b;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = IO::from_float(v[j]);
  }
}

// How the "units" of a call (rows, or the groups of rows) lie on lanes: `lanes` lanes hold a unit
// (8, 16, 32 or 64 of a wave, or the whole workgroup), `segs` units of a workgroup run side by
// side, and the launch's `stride` units advance the row by `drow` and the group by `dg`.
struct UnitLayout {
  int32_t lanes, segs, groups, width;
  int64_t units, stride, drow;
  int32_t dg;
};

// Sum of N values over the lanes of a unit, the same in each of them.  Within 16 lanes the partner
// comes by DPP (its quad neighbours, then mirrored halves and rows), beyond by a shuffle, over the
// waves through LDS: `lds` has 2 N rows of 16 floats, and `phase` alternates between them, so that
// one barrier per sum is enough.  All waves of a workgroup call it together when lanes > 64.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(
                 __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ void unit_sums(float (&v)[N], int lanes, float* lds, int phase) {
#pragma unroll
  for (int q = 0; q < N; ++q) {
    v[q] = dpp_add<0xb1>(v[q]);    // lane ^ 1
    v[q] = dpp_add<0x4e>(v[q]);    // lane ^ 2
    v[q] = dpp_add<0x141>(v[q]);   // the other four of eight
  }
  if (lanes > 8) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = dpp_add<0x140>(v[q]);  // the other eight of sixteen
  }
  if (lanes > 16) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] += __shfl_xor(v[q], 16);
  }
  if (lanes > 32) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] += __shfl_xor(v[q], 32);
  }
  if (lanes > 64) {
    float* at = lds + (phase & 1) * N * 16;
    const int waves = lanes >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int q = 0; q < N; ++q) at[q * 16 + (threadIdx.x >> 6)] = v[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < N; ++q) {
      float s = at[q * 16];
      for (int w = 1; w < waves; ++w) s += at[q * 16 + w];
      v[q] = s;
    }
  }
}

}  // namespace ss
