// ss_mfma.h -- operands of the 16x16x32 bf16 matrix instruction from LDS tiles, fp32 values as
// pairs of bf16, and sums over a wave, for the multi-head scan's kernels.
#pragma once

#include "ss_device.h"

namespace ss {

using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f32x4 = float __attribute__((ext_vector_type(4)));

struct Op {  // one MFMA operand: 8 bf16 in 4 dwords
  uint32_t w[4];
};

__device__ __forceinline__ f32x4 mfma(const Op& a, const Op& b, f32x4 c) {
  using u4 = uint32_t __attribute__((ext_vector_type(4)));
  const u4 av = {a.w[0], a.w[1], a.w[2], a.w[3]};
  const u4 bv = {b.w[0], b.w[1], b.w[2], b.w[3]};
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av),
                                                 __builtin_bit_cast(bf16x8, bv), c, 0, 0, 0);
}

// Two floats to two bf16 (round to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  using b2 = __bf16 __attribute__((ext_vector_type(2)));
  const b2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}
// 8-byte store through a buffer resource (dropped past its range).
__device__ __forceinline__ void store8(uint2 v, rsrc_t r, uint32_t off) {
  using v2u = __attribute__((ext_vector_type(2))) unsigned int;
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u, v), r, off, 0, 0);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Four bf16 of column n0 + l16 (l16 = lane % 16) in rows s0 .. s0 + 3 of a row-major LDS tile
// of `stride` elements per row, as (rows s0, s0 + 1) and (s0 + 2, s0 + 3) pairs: an MFMA operand
// half with K running down a column.  The gfx950 LDS transpose read (ds_read_b64_tr_b16) hands
// lane i of each 16-lane group element i % 4 of the 8 bytes read by lanes i / 4 + 4 m of the
// group, m = 0..3 (lane layout checked on the MI355X); so lane j reads the 4 elements of row
// s0 + j / 4 starting at column n0 + 4 (j % 4).
// The same from a tile whose rows hold their 8-byte units (4 bf16) XOR-permuted by `key`
// (uniform over rows s0 .. s0 + 3): lane j reads logical columns n0 + 4 (j % 4) .. + 3 where the
// permutation put them.
__device__ __forceinline__ uint2 tr_read4_swz(const uint16_t* tile, int stride, int s0, int n0,
                                              int l16, int key) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef v4s __attribute__((address_space(3)))* lds_v4s;
  const int unit = (n0 >> 2) + (l16 & 3);
  const uint16_t* q = tile + (s0 + (l16 >> 2)) * stride + 4 * (unit ^ key);
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(q)));
}
__device__ __forceinline__ uint2 tr_read4(const uint16_t* tile, int stride, int s0, int n0,
                                          int l16) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef v4s __attribute__((address_space(3)))* lds_v4s;
  const uint16_t* q = tile + (s0 + (l16 >> 2)) * stride + n0 + 4 * (l16 & 3);
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(q)));
}

// Split (a, b) into high and low bf16 pairs: a = hi + lo to about 2^-17 relative.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  lo = pack_bf16(a - lo_f(hi), b - hi_f(hi));
}

// Inclusive prefix sum over the 64 lanes of the wave: Hillis-Steele steps inside each 16-lane
// row by DPP row shifts (lanes shifted in from outside the row read 0), then the row totals
// carried across rows by the GFX9 row broadcasts: lane 15 of rows 0 and 2 added to rows 1 and 3,
// then lane 31 (the total of rows 0 and 1) to rows 2 and 3 (rows left out of a row mask add 0).
__device__ __forceinline__ float wave_prefix_sum(float x) {
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x111, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x112, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x114, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x118, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x142, 0xa, 0xf, false));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x143, 0xc, 0xf, false));
  return x;
}

// The operand whose rows (or columns) are r0 + l16 of a row-major tile, K = k0 + 8 g4 + 0..7 along
// them (16-byte aligned).
__device__ __forceinline__ Op op_along(const uint16_t* tile, int stride, int r0, int k0, int l16,
                                       int g4) {
  const uint4 v = *reinterpret_cast<const uint4*>(tile + (r0 + l16) * stride + k0 + 8 * g4);
  return Op{{v.x, v.y, v.z, v.w}};
}
// The operand whose rows (or columns) are the tile's columns c0 + l16, K = k0 + 8 g4 + 0..7 down
// them.
__device__ __forceinline__ Op op_down(const uint16_t* tile, int stride, int k0, int c0, int l16,
                                      int g4) {
  const uint2 k03 = tr_read4(tile, stride, k0 + 8 * g4, c0, l16);
  const uint2 k47 = tr_read4(tile, stride, k0 + 8 * g4 + 4, c0, l16);
  return Op{{k03.x, k03.y, k47.x, k47.y}};
}

}  // namespace ss
