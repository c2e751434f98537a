// ss_gated_fwd.hip -- the gated linear recurrence over a whole sequence.
//
// One workgroup per tile of kWaves x kSteps steps by 64 channels, one channel per lane; wave w owns
// kSteps consecutive steps.  Each lane loads its steps of its channel at once, forms decay and
// input in registers, and reduces them to a Piece; the waves' pieces meet in LDS, the tile's goes
// to the chain (ss_gated_chain.h), and with the state before its first step every wave runs its
// steps again from the registers and stores.  Inputs are read once and outputs written once.
//
// What bounds it: memory.  1 x 262144 x 1536 bfloat16 without a gate moves 3.2 GB in 688 us
// (4.7 TB/s, what a copy of that size reaches); 4 x 4096 x 5120 with a gate 0.84 GB in 182 us
// (4.6 TB/s), the VALU issuing in four fifths of the cycles (44 operations per element, eight of
// them transcendental: two for each of the three sigmoids, the decay and the root).
// Why this tile: a tile pays for the chain, the parameters and the waves' pieces once, so long ones
// are better, as far as registers let two workgroups share a CU.  At 8 x 2048 x 1536, 61 us now, 64
// steps in four or eight waves took 93 and 85 us when 128 took 66 (with two channels per lane 69),
// 96 steps 79, 192 in twelve waves 71, 256 in sixteen 67; 32 steps per wave gained 3 % at
// 1 x 262144 x 1536 and lost 4 % in float32.  Workgroups that stay and draw their next tile early
// took 780 us there, at 710 without.
#include "ss_block.h"
#include "ss_gated_chain.h"

namespace ss {
namespace {

constexpr int kSteps = kGatedFwdSteps;
constexpr int kTile = kGatedFwdTile;
constexpr int kWaves = kTile / kSteps;

// Four waves per SIMD (two workgroups per CU) whatever the registers: told so, the compiler takes
// up to 128 and keeps more loads in flight (708 against 730 us at 1 x 262144 x 1536 when tried).
template <class IO, bool GATE, bool PAST>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(4, 4)))
void gated_fwd_kernel(GatedArgs p, int32_t groups, int32_t nseg, uint32_t log_sets) {
  using elem = typename IO::elem;
  using R = Rows<IO, 1, PAST>;
  using F = Rows<F32, 1>;
  __shared__ Piece pieces[kWaves][64];
  __shared__ float before[64];
  __shared__ slot_t far[kFar * 64];
  __shared__ uint32_t drawn;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t chains = static_cast<uint32_t>(p.batch) * groups;
  const Draw drawn_tile =
      draw_tile(static_cast<uint32_t*>(p.workspace), &drawn, chains, nseg, log_sets);
  if (!drawn_tile.some) return;
  const uint32_t seg = drawn_tile.pos, chain = drawn_tile.chain;
  const int64_t b = chain / groups;
  const int64_t c = static_cast<int64_t>(chain % groups) * 64 + lane;
  const bool active = c < p.d_inner;
  const int64_t t0 = static_cast<int64_t>(seg) * kTile + wave * kSteps;
  // the wave's rows: kSteps of them, or what is left of the sequence (none past its end)
  const int64_t left = p.seqlen - t0;
  const int n = left < 0 ? 0 : left < kSteps ? static_cast<int>(left) : kSteps;
  const int64_t row0 = b * p.seqlen;
  const int64_t first = n ? (row0 + t0) * p.d_inner : 0;
  const uint32_t row = static_cast<uint32_t>(p.d_inner) * sizeof(elem);
  const uint32_t col = active ? static_cast<uint32_t>(c) * sizeof(elem) : kOffNone;
  auto rows = [&](const void* base) { return rows_of<IO, 1, PAST>(base, first, n * row); };
  // Parameters and starts are asked for first: what is waited for last is then the rows, once.
  // (An absent array is an empty resource and reads as zeros, without a branch to wait at.)
  const uint32_t wide = static_cast<uint32_t>(p.d_inner) * 4;
  const uint32_t par_at = active ? static_cast<uint32_t>(c) * 4 : kOffNone;
  auto param = [&](const float* q, int64_t line) {
    return F{make_buf(q + (q ? line * p.d_inner : 0), q ? wide : 0)}.load(par_at);
  };
  const uint8_t begins = __builtin_amdgcn_raw_buffer_load_b8(
      make_buf(p.starts + (p.starts && n ? row0 + t0 : 0), p.starts ? n : 0), lane, 0, 0);
  const float A = kLog2e * param(p.A, 0), rb = -kLog2e * param(p.r_bias, 0),
              ib = -kLog2e * param(p.i_bias, 0);
  float h = param(seg == 0 ? p.h0 : nullptr, b);
  typename R::raw xr[kSteps], rr[kSteps], ir[kSteps], zr[kSteps];
  {
    const R r = rows(p.r), i = rows(p.i), x = rows(p.x);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      rr[j] = r.load(col + j * row);
      ir[j] = i.load(col + j * row);
      xr[j] = x.load(col + j * row);
    }
  }
  const uint32_t fresh = static_cast<uint32_t>(__ballot(begins != 0));  // bit j: step j starts

  // Decay and input of every step.  Rows past the end were read as zeros; their steps are made to
  // change nothing below.
  float a[kSteps], in[kSteps], y = 0.0f;
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const float l = A * sigmoid_biased(IO::widen(rr[j]), rb);
    a[j] = exp2_hw(l);
    in[j] = decay_scale(l, a[j]) * sigmoid_biased(IO::widen(ir[j]), ib) * IO::widen(xr[j]);
    if (j < n) y += l;
  }
  // Starts and the end of the sequence are the exception: one test for the whole wave.
  const bool plain = fresh == 0 && n == kSteps;
  if (n < kSteps) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      a[j] = j < n ? a[j] : 1.0f;
      in[j] = j < n ? in[j] : 0.0f;
    }
  }
  auto step = [&](int j, float s) { return fresh >> j & 1 ? in[j] : fmaf(a[j], s, in[j]); };
  // the product of the decays as 2 to the sum of their exponents
  Piece piece{fresh ? 0.0f : fmaxf(exp2_hw(y), kTinyDecay), 0.0f};
  if (plain) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) piece.H = fmaf(a[j], piece.H, in[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) piece.H = step(j, piece.H);
  }
  if (GATE) {
    const R z = rows(p.z);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) zr[j] = z.load(col + j * row);
  }
  pieces[wave][lane] = piece;
  __syncthreads();

  // The state before the tile: one wave asks the chain, the others wait.
  if (nseg > 1) {
    if (wave == 0) {
      slot_t* slots = reinterpret_cast<slot_t*>(static_cast<char*>(p.workspace) + kChainHead) +
                      static_cast<int64_t>(chain) * 64 + lane;
      const int64_t stride = static_cast<int64_t>(chains) * 64;
      const bool feeds = static_cast<int32_t>(seg) + 1 < nseg;
      Piece whole = piece;
      if (feeds) {
#pragma unroll
        for (int k = 1; k < kWaves; ++k) whole = then(whole, pieces[k][lane]);
        if (seg) publish(slots + seg * stride, whole);
      }
      if (seg) h = look_back(slots, stride, seg, far);
      if (feeds) publish(slots + seg * stride, Piece{0.0f, advance(whole, h)});
      before[lane] = h;
    }
    __syncthreads();
    h = before[lane];
  }
  for (int k = 0; k < wave; ++k) h = advance(pieces[k][lane], h);

  const R o = rows(p.out);
  auto finish = [&](int j) {  // out of step j from its state
    const float out = GATE ? h * silu_f(IO::widen(zr[j])) : h;
    if (p.out) o.store(&out, col + j * row);
  };
  if (plain) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      h = fmaf(a[j], h, in[j]);
      finish(j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      h = step(j, h);
      finish(j);
    }
  }
  // The wave that holds the last step of a chunk or of the sequence (its steps past the end left
  // the state as it was).
  static_assert(SS_GATED_CHUNK % kSteps == 0, "a chunk ends with a wave's last step");
  if (n > 0 && active) {
    if (p.states && (left <= kSteps || (t0 + kSteps) % SS_GATED_CHUNK == 0))
      p.states[(b * p.n_chunks + t0 / SS_GATED_CHUNK) * p.d_inner + c] = h;
    if (p.h_last && left <= kSteps) p.h_last[b * p.d_inner + c] = h;
  }
}

int64_t segments_of(int64_t seqlen) { return (seqlen + kTile - 1) / kTile; }

template <class IO>
hipError_t launch(const GatedArgs& a, hipStream_t stream) {
  const int64_t groups = (a.d_inner + 63) / 64, nseg = segments_of(a.seqlen);
  const int64_t chain = chain_bytes(a.batch, nseg, a.d_inner);
  if (chain) {
    const hipError_t e = launch_zero_bytes(a.workspace, chain, stream);
    if (e != hipSuccess) return e;
  }
  // a sequence shorter than a tile needs fewer waves
  const int waves = nseg > 1 ? kWaves : static_cast<int>((a.seqlen + kSteps - 1) / kSteps);
  const dim3 grid(static_cast<unsigned>(a.batch * groups * nseg)), block(64 * waves);
  const int32_t g = static_cast<int32_t>(groups), n = static_cast<int32_t>(nseg);
  const int64_t row = a.d_inner * sizeof(typename IO::elem);
  const uint32_t log_sets = chain_log_sets(a.batch * groups, nseg, row);
  const int64_t bytes = a.batch * a.seqlen * row;
  auto go = [&](auto gate, auto past) {
    hipLaunchKernelGGL((gated_fwd_kernel<IO, gate, past>), grid, block, 0, stream, a, g, n,
                       log_sets);
  };
  with_bools(go, a.z != nullptr, passes_cache(bytes * (a.z ? 5 : 4), row));
  return hipGetLastError();
}

}  // namespace

size_t gated_fwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner) {
  return static_cast<size_t>(chain_bytes(batch, segments_of(seqlen), d_inner));
}

hipError_t launch_gated_fwd(const GatedArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch<BF16>(a, stream) : launch<F32>(a, stream);
}

}  // namespace ss
