// ss_philox.h -- the counter-based generator behind dropout: Philox4x32-10 (J. K. Salmon,
// M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).
//
// The mask of a (rows, dim) array is a function of the element's place alone: the eight columns
// 8 c .. 8 c + 7 of row r share the four 32-bit words for the counter (c, r, offset), under the key
// `seed`; column 8 c + j takes the j-th 16 bits of them, lowest first.  It is kept where those are
// at least round(65536 p).  Nothing is stored, and every operator that draws from the same (seed,
// offset) for an array of the same shape sees the same mask, so the gradient recomputes it.
//
// Sixteen bits an element, not 32: a call costs about 110 VALU slots (two 32 x 32 multiplies a
// round, at a quarter of the rate), 14 per element of eight, 28 of four.  The price is that p is
// used as a multiple of 2^-16; the scale of what is kept uses that multiple, so the expectation
// stays exact.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ss {

struct PhiloxKey {
  uint32_t seed_lo, seed_hi, off_lo, off_hi;
};

// The two 64-bit numbers at `rng` (uniform: scalar loads).
__device__ __forceinline__ PhiloxKey philox_key(const uint64_t* rng) {
  const uint64_t s = rng[0], o = rng[1];
  return PhiloxKey{static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32),
                   static_cast<uint32_t>(o), static_cast<uint32_t>(o >> 32)};
}

__device__ __forceinline__ uint4 philox(const PhiloxKey& k, uint32_t col8, uint32_t row) {
  uint32_t c0 = col8, c1 = row, c2 = k.off_lo, c3 = k.off_hi, k0 = k.seed_lo, k1 = k.seed_hi;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Which of eight columns are kept, bit j for column j: those whose bits are at least `cut`.
__device__ __forceinline__ uint32_t keep8(const PhiloxKey& k, uint32_t col8, uint32_t row,
                                          uint32_t cut) {
  const uint4 w = philox(k, col8, row);
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
  uint32_t keep = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t bits = j & 1 ? q[j >> 1] >> 16 : q[j >> 1] & 0xffffu;
    keep |= bits >= cut ? 1u << j : 0u;
  }
  return keep;
}

// v times `up` where it is kept, else 0 (chosen, not multiplied: an infinity or a NaN that is
// dropped is gone).
__device__ __forceinline__ void drop8(float (&v)[8], uint32_t keep, float up) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = keep >> j & 1 ? v[j] * up : 0.0f;
}

}  // namespace ss
