// ss_gated_chain.h -- how the workgroups of the gated recurrence hand the state from tile to tile.
//
// A workgroup owns one tile: T steps of one batch row and 64 V channels.  The sequence is a chain
// of tiles per (batch row, channel group); a tile needs the state at its start, which depends on
// every tile before it.  Two passes (summaries, then outputs) would read the inputs twice; here
// each tile is read once: it reduces its steps to a Piece, publishes it, picks up the pieces and
// end states of the tiles before it, and only then runs its steps, which are still in registers.
//
// A slot holds one channel's Piece of one tile in 64 bits: H in the low half, P in the high half
// with the sign bit set (P is never negative).  An empty slot is 0.  An end state is published
// over the piece as the piece (P = 0, H = state): nothing before it matters any more, which is
// just what P = 0 says, so a reader treats it and a piece with a start in it alike.  One relaxed
// 64-bit atomic at device scope carries value and validity together, so no fence is needed (a
// device-scope release would write back the XCD's whole L2).
//
// A tile reads the W tiles before it at once, one per wave, and waits until each holds a piece and
// one of them an end state, then runs from the nearest end state forward.  Every tile's end state
// is formed as advance(piece, state before) whoever forms it, so the result does not depend on
// timing: two runs agree bit for bit.
//
// Tiles are numbered by a counter that workgroups draw from as they start, with the tiles that are
// waited on first.  So a workgroup waits only for ones that are running or done, and every wait
// ends.  Should a slot stay empty all the same (a workspace that two calls share at the same
// time), the wait gives up after kMaxPolls polls and the tile continues from a NaN.
#pragma once

#include "ss_gated_math.h"

namespace ss {

using slot_t = unsigned long long;

// Workspace of a chain: the counter (in the first kChainHead bytes), then the slots
// [segment][batch row][channel group][64 V].  All of it is cleared before the launch.
constexpr int64_t kChainHead = 256;
constexpr int kMaxPolls = 1 << 20;

__device__ __forceinline__ slot_t pack(Piece p) {
  return static_cast<slot_t>(__float_as_uint(p.P) | 0x80000000u) << 32 | __float_as_uint(p.H);
}
__device__ __forceinline__ Piece unpack(slot_t s) {
  return Piece{__uint_as_float(static_cast<uint32_t>(s >> 32) & 0x7fffffffu),
               __uint_as_float(static_cast<uint32_t>(s))};
}
__device__ __forceinline__ void publish(slot_t* s, Piece p) {
  __hip_atomic_store(s, pack(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ slot_t peek(const slot_t* s) {
  return __hip_atomic_load(s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// This workgroup's tile number.  `lds` is written by the first thread and read after a barrier.
__device__ __forceinline__ uint32_t draw_tile(uint32_t* counter, uint32_t* lds) {
  if (threadIdx.x == 0)
    *lds = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*lds);
}

// The state before tile `pos` of a chain (pos >= 1 tiles come before it), for V channels per
// lane.  `slots` points at this lane's first channel in tile 0 of the chain and `stride` slots lie
// between tiles.  Called by every wave of the workgroup; `look` holds W = blockDim / 64 rows.
template <int V>
__device__ __forceinline__ void state_before(const slot_t* slots, int64_t stride, int64_t pos,
                                             slot_t* look, float* state) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int n = pos < waves ? static_cast<int>(pos) : waves;  // tiles looked at
  const slot_t* mine = slots + (pos - 1 - wave) * stride;
  const slot_t lost = pack(Piece{0.0f, __builtin_nanf("")});
  int polls = 0;                       // this wave's
  for (int round = 0;; ++round) {      // the same in every wave: all see the same `look`
    if (wave < n) {
      slot_t s[V];
      for (;;) {
        bool full = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          s[v] = peek(mine + v);
          full &= s[v] != 0;
        }
        if (__all(full)) break;
        if (++polls > kMaxPolls) {
#pragma unroll
          for (int v = 0; v < V; ++v) s[v] = lost;
          break;
        }
        __builtin_amdgcn_s_sleep(1);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) look[(wave * V + v) * 64 + lane] = s[v];
    }
    __syncthreads();
    // from the farthest tile looked at to the nearest; known from the first end state on
    bool known[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      known[v] = false;
      state[v] = 0.0f;
    }
    for (int k = n - 1; k >= 0; --k) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Piece p = unpack(look[(k * V + v) * 64 + lane]);
        known[v] |= p.P == 0.0f;
        state[v] = advance(p, state[v]);
      }
    }
    bool all = true;
#pragma unroll
    for (int v = 0; v < V; ++v) all &= known[v];
    if (__all(all)) return;
    if (round >= kMaxPolls) {
#pragma unroll
      for (int v = 0; v < V; ++v) state[v] = known[v] ? state[v] : __builtin_nanf("");
      return;
    }
    __syncthreads();  // every wave has read `look` before it is written again
  }
}

}  // namespace ss
