// ss_gated_chain.h -- how the workgroups of the gated recurrence hand the state from tile to tile.
//
// A workgroup owns one tile: T steps of one batch row and 64 channels, one per lane.  The sequence
// is a chain of tiles per (batch row, channel group); a tile needs the state at its start, which
// depends on every tile before it.  Two passes (summaries, then outputs) would read the inputs
// twice; here each tile is read once: it reduces its steps to a Piece, publishes it, picks up the
// pieces and end states of the tiles before it, and only then runs its steps, which are still in
// registers.
//
// A slot holds one channel's Piece of one tile in 64 bits: H in the low half, P in the high half
// with the sign bit set (P is never negative).  An empty slot is 0.  An end state is published
// over the piece as the piece (P = 0, H = state): nothing before it matters any more, which is
// just what P = 0 says, so a reader treats it and a piece with a start in it alike.  One relaxed
// 64-bit atomic at device scope carries value and validity together, so no fence is needed (a
// device-scope release would write back the XCD's whole L2).
//
// One wave of the workgroup reads the kNear tiles before its own at once, until there is an end
// state among them and a piece in every slot nearer than it, then runs forward from that state.
// Where all of them hold pieces but none an end state twice over (few chains, and so many tiles of
// each at work at the same time), it reaches up to kFar tiles back, kMore at a time, through LDS.
// Measured (each comparison here timed in turn, with the kernels as they then stood): 4 near tiles
// against 8 or 12 read every time, 67 against 68 and 69 us at 8 x 2048 x 1536 and 702 against 743
// and 760 us at 1 x 262144 x 1536; the far ones with and without, 91 and 176 us at 1 x 131072 x 64
// (one chain of 1024 tiles), 168 and 220 us at 1 x 131072 x 512, and asked for at once, 769 us at
// 1 x 262144 x 1536.
// Every tile's end state is formed as advance(piece, state before) whoever forms it, so the result
// does not depend on timing: two runs agree bit for bit.
//
// Tiles are numbered by counters that workgroups draw from as they start, with the tiles that are
// waited on first.  So a workgroup waits only for ones that are running or done, and every wait
// ends.  Should a slot stay empty all the same (a workspace that two calls share at the same
// time), the wait gives up after kMaxPolls polls and the tile continues from a NaN.
#pragma once

#include "ss_gated_math.h"

namespace ss {

using slot_t = unsigned long long;

// Workspace of a launch: the counters (in the first kChainHead bytes, a cache line each), then the
// slots [segment][batch row][channel group][64].  All of it is cleared before the launch.
constexpr int64_t kChainHead = 1024;
constexpr int kLogSets = 3, kCounterStep = 32;
inline int64_t chain_bytes(int64_t batch, int64_t segments, int64_t d_inner) {
  if (segments <= 1) return 0;
  return kChainHead + batch * segments * ((d_inner + 63) / 64 * 64) * 8;
}
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

// The chains are dealt to one counter or to eight (sets), in runs of neighbours, and a set's tiles
// are numbered segment by segment.  Workgroups start at the sets in turn, so that a set is an
// XCD's and neighbours, which share cache lines where rows are not whole lines, meet in one L2; one
// whose set has no tile left goes on to the next.  There are as many workgroups as tiles.
struct Draw {
  uint32_t pos, chain;  // the tile's place in its chain, and the chain
  bool some;            // false: none was left (the counters were not clear)
};
// The chains before set `s`.
__device__ __forceinline__ uint32_t share(uint32_t chains, uint32_t s, uint32_t log_sets) {
  return static_cast<uint32_t>(static_cast<uint64_t>(chains) * s >> log_sets);
}
// `lds` is written by the first thread and read after a barrier.
__device__ __forceinline__ Draw draw_tile(uint32_t* counters, uint32_t* lds, uint32_t chains,
                                          uint32_t segments, uint32_t log_sets) {
  if (segments == 1) return Draw{0, blockIdx.x, true};
  const uint32_t last = (1u << log_sets) - 1;
  uint32_t set = blockIdx.x & last;
  for (uint32_t tries = 0;;) {
    if (threadIdx.x == 0)
      *lds = __hip_atomic_fetch_add(counters + set * kCounterStep, 1u, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
    uint32_t first = 0, mine = chains;
    if (log_sets) {
      first = share(chains, set, log_sets);
      mine = share(chains, set + 1, log_sets) - first;
    }
    __syncthreads();
    const uint32_t tile = __builtin_amdgcn_readfirstlane(*lds);
    if (__builtin_expect(tile < mine * segments, 1))
      return Draw{tile / mine, first + tile % mine, true};
    if (tries++ == last) return Draw{0, 0, false};
    set = (set + 1) & last;
    __syncthreads();
  }
}
// Sets of a launch, as a power of two.  Eight where all tiles start at once, two workgroups per CU
// (a single counter serves them one after the other, the last of 512 some 3 us late), and where
// chains are short (one / eight, forward: 8 x 2048 x 1536 63.9 / 60.2 us, 4 x 4096 x 5120 186 /
// 182; training step: 3 x 1111 x 1027 51.4 / 45.5).  In long ones the sets drift apart and take the
// rows of one step at different times, and DRAM pages with them (1 x 262144 x 1536 695 / 797 us;
// 2 x 16384 x 1536 float32 172 / 175), which rows that are not whole lines outweigh a little longer
// (2 x 16384 x 1601 153 / 145, 1 x 65536 x 1537 279 / 297).
inline uint32_t chain_log_sets(int64_t chains, int64_t segments, int64_t row) {
  if (chains < 1 << kLogSets) return 0;
  const int64_t longest = row % 128 == 0 ? 32 : 128;
  return chains * segments <= 512 || segments <= longest ? kLogSets : 0;
}

// The state before tile `pos` >= 1 of a chain, for this lane's channel.  `slots` points at the
// channel in tile 0 of the chain and `stride` slots lie between tiles.  For one wave; `far` is LDS
// of its own, kFar rows of 64.
constexpr int kNear = 4, kMore = 8, kFar = kNear + 4 * kMore;
__device__ __forceinline__ float look_back(const slot_t* slots, int64_t stride, int64_t pos,
                                           slot_t* far) {
  const int lane = threadIdx.x & 63;
  const slot_t* nearest = slots + (pos - 1) * stride;
  // slot of the tile k + 1 tiles back (past tile 0, tile 0: its slot only ever holds an end state)
  auto slot = [&](int64_t k) { return peek(nearest - (k < pos ? k : pos - 1) * stride); };
  for (int poll = 0; poll < kMaxPolls; ++poll) {
    slot_t s[kNear];
#pragma unroll
    for (int k = 0; k < kNear; ++k) s[k] = slot(k);
    bool known = false, full = true;
    float state = 0.0f;
#pragma unroll
    for (int k = kNear - 1; k >= 0; --k) {
      const Piece p = unpack(s[k]);
      known = s[k] != 0 && (known || p.P == 0.0f);
      full &= s[k] != 0;
      state = advance(p, state);
    }
    if (__all(known)) return state;
    if (poll >= 2 && __all(full)) {
#pragma unroll
      for (int k = 0; k < kNear; ++k) far[k * 64 + lane] = s[k];
      int depth = kNear;
      while (depth < kFar && depth < pos) {
        slot_t f[kMore];
#pragma unroll
        for (int k = 0; k < kMore; ++k) f[k] = slot(depth + k);
        bool gap = false;  // an empty slot before any end state
#pragma unroll
        for (int k = 0; k < kMore; ++k) {
          far[(depth + k) * 64 + lane] = f[k];
          gap |= f[k] == 0 && !known;
          known |= !gap && unpack(f[k]).P == 0.0f;
        }
        depth += kMore;
        if (__any(gap)) break;
        if (__all(known)) {
          float h = 0.0f;
          for (int k = depth - 1; k >= 0; --k) h = advance(unpack(far[k * 64 + lane]), h);
          return h;
        }
      }
    }
    __builtin_amdgcn_s_sleep(1);
  }
  return __builtin_nanf("");
}

}  // namespace ss
