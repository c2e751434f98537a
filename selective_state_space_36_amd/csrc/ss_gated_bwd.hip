// ss_gated_bwd.hip -- gradients of the gated linear recurrence.
//
// Tiles of kWaves x kSteps = SS_GATED_CHUNK steps by 64 channels, one workgroup each, so that the
// state before a tile is a saved one.  Each lane loads its steps of x, r, i, dout (and z) once.
// The states inside the tile come from the waves' pieces, as in the forward.  The adjoint runs the
// other way: with c_t = a_t lam_t the value that step t hands to step t - 1,
// c_t = a_t (g_t + c_{t+1}), so a piece of steps maps the value entering at its right end to the
// one leaving at its left as c -> P c + M with the same product P.  Tiles are chained from the
// last to the first.  The sums over tokens are added per lane over the steps, over the waves in
// LDS, and over the tiles by a second kernel, always in the same order.
//
// What bounds it: memory and its latency.  4 x 4096 x 5120 bfloat16 with a gate moves 1.55 GB in
// 340 us (4.6 TB/s; a copy of that size reaches 4.9); without the wait for the chain it took 4 %
// less, with 20 % fewer VALU operations 1 % less.
// Why eight steps per wave in eight waves: sixteen hold too many registers for two workgroups on
// a CU, and chunks of 32 and 128 steps took 714 and 612 us a training step against then 566.  Two
// channels per lane spill (874 us).
#include "ss_block.h"
#include "ss_gated_chain.h"

namespace ss {
namespace {

constexpr int kSteps = kGatedBwdSteps;
constexpr int kTile = SS_GATED_CHUNK;  // so that a tile starts at a saved state
constexpr int kWaves = kTile / kSteps;

template <class IO, bool GATE, bool PAST>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(4, 4)))
void gated_bwd_kernel(GatedArgs p, const float* states, float* part, int32_t groups,
                      int32_t nseg, uint32_t log_sets) {
  using elem = typename IO::elem;
  using R = Rows<IO, 1, PAST>;
  using F = Rows<F32, 1>;
  __shared__ Piece pieces[kWaves][64];
  __shared__ float back[kWaves][64];
  __shared__ float after[64];
  __shared__ float sums[3][kWaves][64];
  __shared__ slot_t far[kFar * 64];
  __shared__ uint32_t drawn;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const uint32_t chains = static_cast<uint32_t>(p.batch) * groups;
  const Draw drawn_tile =
      draw_tile(static_cast<uint32_t*>(p.workspace), &drawn, chains, nseg, log_sets);
  if (!drawn_tile.some) return;
  const uint32_t pos = drawn_tile.pos, chain = drawn_tile.chain;  // pos 0 is the last segment
  const uint32_t seg = nseg - 1 - pos;
  const int64_t b = chain / groups;
  const int64_t c = static_cast<int64_t>(chain % groups) * 64 + lane;
  const bool active = c < p.d_inner;
  const int64_t t0 = static_cast<int64_t>(seg) * kTile + wave * kSteps;
  const int64_t row0 = b * p.seqlen;
  // the wave's rows: kSteps of them, or what is left of the sequence (none past its end)
  const int64_t left = p.seqlen - t0;
  const int n = left < 0 ? 0 : left < kSteps ? static_cast<int>(left) : kSteps;
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
  float h = param(seg ? states : p.h0, seg ? b * p.n_chunks + seg - 1 : b);
  float carry = param(pos == 0 ? p.dh_last : nullptr, b);
  typename R::raw xr[kSteps], rr[kSteps], ir[kSteps], gr[kSteps], zr[kSteps];
  {
    const R r = rows(p.r), i = rows(p.i), x = rows(p.x), u = rows(p.dout), z = rows(p.z);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      rr[j] = r.load(col + j * row);
      ir[j] = i.load(col + j * row);
      xr[j] = x.load(col + j * row);
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      gr[j] = u.load(col + j * row);
      if (GATE) zr[j] = z.load(col + j * row);
    }
  }
  const uint32_t fresh = static_cast<uint32_t>(__ballot(begins != 0));  // bit j: step j starts

  // Decays and gates of every step.  Rows past the end were read as zeros; their steps are made
  // to change nothing.
  float a[kSteps], s[kSteps], rs[kSteps], rg[kSteps], ig[kSteps], y = 0.0f;
  float hp[kSteps];  // the input term, then the state before the step
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    rg[j] = sigmoid_biased(IO::widen(rr[j]), rb);
    ig[j] = sigmoid_biased(IO::widen(ir[j]), ib);
    const float l = A * rg[j];
    a[j] = exp2_hw(l);
    // 1 / s from one reciprocal root, and s from it; both 0 where s^2 is 0 or too small for the
    // root's unit (which takes it for 0 and returns infinity), but not where it is NaN
    const float v = one_minus_square(l, a[j]);
    rs[j] = fabsf(v) < kTinyDecay ? 0.0f : rsq_hw(v);
    s[j] = v * rs[j];
    hp[j] = s[j] * ig[j] * IO::widen(xr[j]);
    y += l;
  }
  // Starts and the end of the sequence are the exception: one test for the whole wave.
  const bool plain = fresh == 0 && n == kSteps;
  if (n < kSteps) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      a[j] = j < n ? a[j] : 1.0f;
      hp[j] = j < n ? hp[j] : 0.0f;
    }
  }
  Piece piece{0.0f, 0.0f};
  if (plain) {
    piece.P = fmaxf(exp2_hw(y), kTinyDecay);  // the decays' product: 2 to the sum of exponents
#pragma unroll
    for (int j = 0; j < kSteps; ++j) piece.H = fmaf(a[j], piece.H, hp[j]);
  } else {
    if (!fresh) {
      piece.P = 1.0f;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) piece.P = fmaxf(piece.P * a[j], kTinyDecay);
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      piece.H = fresh >> j & 1 ? hp[j] : fmaf(a[j], piece.H, hp[j]);
  }
  pieces[wave][lane] = piece;
  __syncthreads();
  for (int k = 0; k < wave; ++k) h = advance(pieces[k][lane], h);

  // the states before each step, the gated upstream gradient, dz, and the adjoint's piece
  float g[kSteps], M = 0.0f;
  const R dzr = rows(p.dz);
  auto forward = [&](int j, bool drop) {
    if (drop) h = 0.0f;
    const float in = hp[j];
    hp[j] = h;
    h = fmaf(a[j], h, in);
    g[j] = IO::widen(gr[j]);
    if (GATE) {
      const float z = IO::widen(zr[j]), sg = sigmoid_f(z);
      const float silu = z * sg;
      const float dz = g[j] * h * fmaf(silu, 1.0f - sg, sg);
      dzr.store(&dz, col + j * row);
      g[j] *= silu;
    }
  };
  if (plain) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) forward(j, false);
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) M = a[j] * (g[j] + M);
  } else {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) forward(j, fresh >> j & 1);
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) M = fresh >> j & 1 ? 0.0f : a[j] * (g[j] + M);
  }
  back[wave][lane] = M;
  __syncthreads();

  // The value entering at the tile's right end: one wave asks the chain, the others wait.
  if (nseg > 1) {
    if (wave == 0) {
      slot_t* slots = reinterpret_cast<slot_t*>(static_cast<char*>(p.workspace) + kChainHead) +
                      static_cast<int64_t>(chain) * 64 + lane;
      const int64_t stride = static_cast<int64_t>(chains) * 64;
      Piece whole{pieces[kWaves - 1][lane].P, back[kWaves - 1][lane]};
      if (seg) {
#pragma unroll
        for (int k = kWaves - 2; k >= 0; --k)
          whole = then(whole, Piece{pieces[k][lane].P, back[k][lane]});
        if (pos) publish(slots + pos * stride, whole);
      }
      if (pos) carry = look_back(slots, stride, pos, far);
      if (seg) publish(slots + pos * stride, Piece{0.0f, advance(whole, carry)});
      after[lane] = carry;
    }
    __syncthreads();
    carry = after[lane];
  }
  for (int k = waves - 1; k > wave; --k)
    carry = advance(Piece{pieces[k][lane].P, back[k][lane]}, carry);

  const R dxr = rows(p.dx), drr = rows(p.dr), dir = rows(p.di);
  float sum_A = 0.0f, sum_r = 0.0f, sum_i = 0.0f;
  auto gradients = [&](int j, bool drop) {
    const float x = IO::widen(xr[j]);
    const float lam = g[j] + carry;
    carry = drop ? 0.0f : a[j] * lam;
    const float w = ig[j] * x;
    // a h - ig x a^2 / s, whose second term is 0 where s = 0: there a = 1, and dx, di vanish too
    const float dl = lam * (a[j] * fmaf(-w * rs[j], a[j], hp[j]));
    const float ls = lam * s[j], q = dl * rg[j];
    const float dx = ls * ig[j];
    const float dr = q * (kLn2 * A) * (1.0f - rg[j]);
    const float di = ls * w * (1.0f - ig[j]);
    sum_A += q;
    sum_r += dr;
    sum_i += di;
    dxr.store(&dx, col + j * row);
    drr.store(&dr, col + j * row);
    dir.store(&di, col + j * row);
  };
  if (plain) {
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) gradients(j, false);
  } else {
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      if (j < n) gradients(j, fresh >> j & 1);
    }
  }
  if (p.dh0 && seg == 0 && wave == 0 && active) p.dh0[b * p.d_inner + c] = carry;
  // the tile's sums: one row of part per tile, [3][batch * nseg][d_inner]
  sums[0][wave][lane] = sum_A;
  sums[1][wave][lane] = sum_r;
  sums[2][wave][lane] = sum_i;
  __syncthreads();
  for (int q = wave; q < 3; q += waves) {
    float acc = sums[q][0][lane];
    for (int k = 1; k < waves; ++k) acc += sums[q][k][lane];
    if (active) part[(q * p.batch * nseg + b * nseg + seg) * p.d_inner + c] = acc;
  }
}

int64_t segments_of(int64_t seqlen) { return (seqlen + kTile - 1) / kTile; }

// Workspace: the chain (also the one of the pass that recomputes the states), the tiles' sums,
// and the states when they are recomputed.
struct Layout {
  int64_t chain, part, states, total;  // bytes of the chain to clear; byte offsets
};
Layout layout(int64_t batch, int64_t seqlen, int64_t d_inner, bool given) {
  const int64_t nseg = segments_of(seqlen);
  Layout l;
  l.chain = chain_bytes(batch, nseg, d_inner);
  int64_t head = l.chain;
  if (!given) {
    const int64_t f = static_cast<int64_t>(gated_fwd_ws_bytes(batch, seqlen, d_inner));
    head = head > f ? head : f;
  }
  l.part = (head + 255) / 256 * 256;
  l.states = l.part + (3 * batch * nseg * d_inner * 4 + 255) / 256 * 256;
  l.total = l.states + (given ? 0 : batch * nseg * d_inner * 4);
  return l;
}

template <class IO>
hipError_t launch(const GatedArgs& a, const Layout& l, const float* states, float* part,
                  hipStream_t stream) {
  const int64_t groups = (a.d_inner + 63) / 64, nseg = segments_of(a.seqlen);
  if (l.chain) {
    const hipError_t e = launch_zero_bytes(a.workspace, l.chain, stream);
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
    hipLaunchKernelGGL((gated_bwd_kernel<IO, gate, past>), grid, block, 0, stream, a, states, part,
                       g, n, log_sets);
  };
  with_bools(go, a.z != nullptr, passes_cache(bytes * (a.z ? 9 : 7), row));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t tiles = a.batch * nseg, plane = tiles * a.d_inner;
  ColumnSums c{};
  c.lines = tiles;
  c.stride = c.cols = a.d_inner;
  c.add(part, a.dA, 1);
  c.add(part + plane, a.dr_bias, 1);
  c.add(part + 2 * plane, a.di_bias, 1);
  return launch_column_sums(c, stream);
}

}  // namespace

size_t gated_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, bool given) {
  return static_cast<size_t>(layout(batch, seqlen, d_inner, given).total);
}

hipError_t launch_gated_bwd(const GatedArgs& a, bool bf16, hipStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  const Layout l = layout(a.batch, a.seqlen, a.d_inner, a.states != nullptr);
  const float* states = a.states;
  float* part = reinterpret_cast<float*>(ws + l.part);
  if (!states) {
    GatedArgs f = a;
    f.z = nullptr;
    f.out = nullptr;
    f.h_last = nullptr;
    f.states = reinterpret_cast<float*>(ws + l.states);
    states = f.states;
    const hipError_t e = launch_gated_fwd(f, bf16, stream);
    if (e != hipSuccess) return e;
  }
  return bf16 ? launch<BF16>(a, l, states, part, stream) : launch<F32>(a, l, states, part, stream);
}

}  // namespace ss
