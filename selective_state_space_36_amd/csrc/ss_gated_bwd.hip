// ss_gated_bwd.hip -- gradients of the gated linear recurrence.
//
// The tiles are the forward's: kWaves x kSteps steps by 64 V channels, one workgroup each, with
// kTile = SS_GATED_CHUNK, so the state before a tile is a saved one.  Each lane loads its steps of
// x, r, i, dout (and z) once.  The states inside the tile come from the waves' pieces, as in the
// forward.  The adjoint runs the other way: with c_t = a_t lam_t the value that step t hands to
// step t - 1, c_t = a_t (g_t + c_{t+1}), so a piece of steps maps the value entering at its right
// end to the one leaving at its left as c -> P c + M with the same product P.  Tiles are chained
// from the last to the first.  The sums over tokens are added per lane over the steps, over the
// waves in LDS, and over the tiles by a second kernel, always in the same order.
#include "ss_block.h"
#include "ss_gated_chain.h"

namespace ss {
namespace {

constexpr int kSteps = 8;
constexpr int kWaves = 8;
constexpr int kTile = kSteps * kWaves;
static_assert(kTile == SS_GATED_CHUNK, "a tile starts at a saved state");

template <class IO, int V, bool GATE, bool PACKED>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(4)))
void gated_bwd_kernel(GatedArgs p, const float* states, float* part, int32_t groups,
                      int32_t nseg) {
  using elem = typename IO::elem;
  using L = Lanes<IO, V>;
  __shared__ Piece pieces[kWaves][V][64];
  __shared__ float back[kWaves][V][64];
  __shared__ slot_t look[kWaves * V * 64];
  __shared__ uint32_t drawn;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const uint32_t chains = static_cast<uint32_t>(p.batch) * groups;
  const uint32_t tile =
      nseg > 1 ? draw_tile(static_cast<uint32_t*>(p.workspace), &drawn) : blockIdx.x;
  const uint32_t pos = tile / chains, chain = tile % chains;  // pos 0 is the last segment
  const uint32_t seg = nseg - 1 - pos;
  const int64_t b = chain / groups;
  const int64_t c0 = static_cast<int64_t>(chain % groups) * (64 * V) + lane * V;
  const bool active = c0 < p.d_inner;
  const int64_t c = active ? c0 : 0;
  const int64_t t0 = static_cast<int64_t>(seg) * kTile + wave * kSteps;
  const int64_t row0 = b * p.seqlen;
  // the wave's rows: kSteps of them, or what is left of the sequence (none past its end)
  const int64_t left = p.seqlen - t0;
  const int n = left < 0 ? 0 : left < kSteps ? static_cast<int>(left) : kSteps;
  const int64_t first = n ? (row0 + t0) * p.d_inner : 0;
  const uint32_t row = static_cast<uint32_t>(p.d_inner) * sizeof(elem);
  const uint32_t col = active ? static_cast<uint32_t>(c) * sizeof(elem) : kOffNone;
  auto rows = [&](const void* base) { return rows_of<IO, V>(base, first, n * row); };

  typename L::raw xr[kSteps], rr[kSteps], ir[kSteps], gr[kSteps], zr[kSteps];
  {
    const Rows<IO, V> R = rows(p.r), I = rows(p.i), X = rows(p.x);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      rr[j] = R.load(col + j * row);
      ir[j] = I.load(col + j * row);
      xr[j] = X.load(col + j * row);
    }
    const Rows<IO, V> G = rows(p.dout), Z = rows(p.z);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      gr[j] = G.load(col + j * row);
      if (GATE) zr[j] = Z.load(col + j * row);
    }
  }
  uint32_t fresh = 0;  // bit j: a sequence starts at step j
  if (PACKED) fresh = static_cast<uint32_t>(__ballot(lane < n && p.starts[row0 + t0 + lane]));
  float A[V], rb[V], ib[V], h[V], carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = p.A[c + v];
    rb[v] = p.r_bias ? p.r_bias[c + v] : 0.0f;
    ib[v] = p.i_bias ? p.i_bias[c + v] : 0.0f;
    const int64_t ch = b * p.d_inner + c + v;
    h[v] = seg ? states[(b * p.n_chunks + seg - 1) * p.d_inner + c + v] : p.h0 ? p.h0[ch] : 0.0f;
    carry[v] = pos == 0 && p.dh_last ? p.dh_last[ch] : 0.0f;
  }

  float a[kSteps][V], rg[kSteps][V], ig[kSteps][V];
  float hp[kSteps][V];  // the input term, then the state before the step
  Piece piece[V];
#pragma unroll
  for (int v = 0; v < V; ++v) piece[v] = Piece{1.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const bool beyond = j >= n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      rg[j][v] = sigmoid_f(L::get(rr[j], v) + rb[v]);
      ig[j][v] = sigmoid_f(L::get(ir[j], v) + ib[v]);
      const Decay k = decay_f(A[v] * rg[j][v]);
      a[j][v] = beyond ? 1.0f : fmaxf(k.a, kTinyDecay);
      const float in = beyond ? 0.0f : k.s * ig[j][v] * L::get(xr[j], v);
      hp[j][v] = in;
      const bool cut = PACKED && (fresh >> j & 1);
      piece[v].H = cut ? in : fmaf(a[j][v], piece[v].H, in);
      piece[v].P = fmaxf(piece[v].P * a[j][v], kTinyDecay);
    }
  }
  if (PACKED && fresh) {
#pragma unroll
    for (int v = 0; v < V; ++v) piece[v].P = 0.0f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) pieces[wave][v][lane] = piece[v];
  __syncthreads();
  for (int k = 0; k < wave; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = advance(pieces[k][v][lane], h[v]);
  }

  // the states before each step, the gated upstream gradient, and dz
  float g[kSteps][V];
  const Rows<IO, V> DZ = rows(p.dz);
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const bool beyond = j >= n;
    float dz[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (PACKED && (fresh >> j & 1)) h[v] = 0.0f;
      const float in = hp[j][v];
      hp[j][v] = h[v];
      h[v] = fmaf(a[j][v], h[v], in);
      g[j][v] = L::get(gr[j], v);
      if (GATE) {
        const float z = L::get(zr[j], v), sg = sigmoid_f(z);
        dz[v] = g[j][v] * h[v] * (sg * fmaf(z, 1.0f - sg, 1.0f));
        g[j][v] *= z * sg;
      }
      if (beyond) g[j][v] = 0.0f;
    }
    if (GATE) DZ.store(dz, col + j * row);
  }

  // the waves' adjoint pieces, the tile's, and the value entering at this wave's right end
  float M[V];
#pragma unroll
  for (int v = 0; v < V; ++v) M[v] = 0.0f;
#pragma unroll
  for (int j = kSteps - 1; j >= 0; --j) {
    const bool cut = PACKED && (fresh >> j & 1);
#pragma unroll
    for (int v = 0; v < V; ++v) M[v] = cut ? 0.0f : a[j][v] * (g[j][v] + M[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) back[wave][v][lane] = M[v];
  __syncthreads();
  auto adjoint = [&](int k, int v) { return Piece{pieces[k][v][lane].P, back[k][v][lane]}; };
  if (nseg > 1) {
    Piece whole[V];
    slot_t* slots = reinterpret_cast<slot_t*>(static_cast<char*>(p.workspace) + kChainHead) +
                    static_cast<int64_t>(chain) * (64 * V) + lane * V;
    const int64_t stride = static_cast<int64_t>(chains) * (64 * V);
    const bool feeds = wave == 0 && seg > 0;
    if (feeds) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        whole[v] = adjoint(waves - 1, v);
        for (int k = waves - 2; k >= 0; --k) whole[v] = then(whole[v], adjoint(k, v));
        if (pos) publish(slots + pos * stride + v, whole[v]);
      }
    }
    if (pos) state_before<V>(slots, stride, pos, look, carry);
    if (feeds) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        publish(slots + pos * stride + v, Piece{0.0f, advance(whole[v], carry[v])});
    }
  }
  for (int k = waves - 1; k > wave; --k) {
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = advance(adjoint(k, v), carry[v]);
  }

  const Rows<IO, V> DX = rows(p.dx), DR = rows(p.dr), DI = rows(p.di);
  float sum[3][V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum[0][v] = sum[1][v] = sum[2][v] = 0.0f;
#pragma unroll
  for (int j = kSteps - 1; j >= 0; --j) {
    if (j < n) {
      const bool cut = PACKED && (fresh >> j & 1);
      float dx[V], dr[V], di[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = L::get(xr[j], v);
        const float lam = g[j][v] + carry[v];
        carry[v] = cut ? 0.0f : a[j][v] * lam;
        // s is formed again rather than kept: 16 registers less (the empty statement hides from
        // the compiler that it had it before)
        asm("" : "+v"(rg[j][v]));
        const float s = decay_scale(A[v] * rg[j][v], a[j][v]);
        // a^2 / s, 0 where s = 0: there a = 1 and dx, di vanish too
        const float slope = s > 0.0f ? a[j][v] * a[j][v] * rcp_hw(s) : 0.0f;
        const float w = ig[j][v] * x;
        const float dl = lam * fmaf(a[j][v], hp[j][v], -w * slope);
        dx[v] = lam * s * ig[j][v];
        dr[v] = dl * A[v] * rg[j][v] * (1.0f - rg[j][v]);
        di[v] = lam * s * w * (1.0f - ig[j][v]);
        sum[0][v] = fmaf(dl, rg[j][v], sum[0][v]);
        sum[1][v] += dr[v];
        sum[2][v] += di[v];
      }
      DX.store(dx, col + j * row);
      DR.store(dr, col + j * row);
      DI.store(di, col + j * row);
    }
  }
  if (p.dh0 && seg == 0 && wave == 0 && active) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.dh0[b * p.d_inner + c + v] = carry[v];
  }
  // the tile's sums: one row of part per tile, [3][batch * nseg][d_inner]
  __syncthreads();
  float* red = &back[0][0][0];  // kWaves x V x 64, one quantity at a time
#pragma unroll
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int v = 0; v < V; ++v) red[(wave * V + v) * 64 + lane] = sum[q][v];
    __syncthreads();
    if (wave == 0 && active) {
      const int64_t rows = p.batch * nseg;
      float* o = part + (q * rows + b * nseg + seg) * p.d_inner + c;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float acc = red[v * 64 + lane];
        for (int k = 1; k < waves; ++k) acc += red[(k * V + v) * 64 + lane];
        o[v] = acc;
      }
    }
    __syncthreads();
  }
}

// Sums of the tiles' rows per channel: 16 row strands by 16 channels per workgroup, then the
// strands in order.
__global__ __launch_bounds__(256) void gated_reduce_kernel(GatedArgs p, const float* part,
                                                           int64_t rows) {
  __shared__ float lds[16][17];
  const int q = blockIdx.y;
  float* out = q == 0 ? p.dA : q == 1 ? p.dr_bias : p.di_bias;
  if (!out) return;
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int64_t d = blockIdx.x * 16ll + x;
  float acc = 0.0f;
  if (d < p.d_inner) {
    const float* src = part + q * rows * p.d_inner + d;
    for (int64_t r = y; r < rows; r += 16) acc += src[r * p.d_inner];
  }
  lds[y][x] = acc;
  __syncthreads();
  if (y == 0 && d < p.d_inner) {
    float s = lds[0][x];
    for (int k = 1; k < 16; ++k) s += lds[k][x];
    out[d] = s;
  }
}

int64_t segments_of(int64_t seqlen) { return (seqlen + kTile - 1) / kTile; }

// Workspace: the chain (also the one of the pass that recomputes the states), the tiles' sums,
// and the states when they are recomputed.
struct Layout {
  int64_t part, states, total;  // byte offsets
};
Layout layout(int64_t batch, int64_t seqlen, int64_t d_inner, bool bf16, bool given) {
  const int64_t nseg = segments_of(seqlen), width = (d_inner + 127) / 128 * 128;
  int64_t chain = nseg > 1 ? kChainHead + batch * nseg * width * int64_t(sizeof(slot_t)) : 0;
  if (!given) {
    const int64_t f = static_cast<int64_t>(gated_fwd_ws_bytes(batch, seqlen, d_inner, bf16));
    chain = chain > f ? chain : f;
  }
  Layout l;
  l.part = (chain + 255) / 256 * 256;
  l.states = l.part + (3 * batch * nseg * d_inner * 4 + 255) / 256 * 256;
  l.total = l.states + (given ? 0 : batch * nseg * d_inner * 4);
  return l;
}

template <class IO, int V>
hipError_t launch(const GatedArgs& a, const float* states, float* part, hipStream_t stream) {
  const int64_t groups = (a.d_inner + 64 * V - 1) / (64 * V);
  const int64_t nseg = segments_of(a.seqlen);
  const int64_t tiles = a.batch * groups * nseg;
  if (nseg > 1) {
    const int64_t bytes = kChainHead + tiles * (64 * V) * static_cast<int64_t>(sizeof(slot_t));
    const hipError_t e = launch_zero(static_cast<float*>(a.workspace), bytes / 4, stream);
    if (e != hipSuccess) return e;
  }
  const int waves = nseg > 1 ? kWaves : static_cast<int>((a.seqlen + kSteps - 1) / kSteps);
  const dim3 grid(static_cast<unsigned>(tiles)), block(64 * waves);
  const int32_t g = static_cast<int32_t>(groups), n = static_cast<int32_t>(nseg);
  if (a.z) {
    if (a.starts)
      hipLaunchKernelGGL((gated_bwd_kernel<IO, V, true, true>), grid, block, 0, stream, a, states,
                         part, g, n);
    else
      hipLaunchKernelGGL((gated_bwd_kernel<IO, V, true, false>), grid, block, 0, stream, a,
                         states, part, g, n);
  } else {
    if (a.starts)
      hipLaunchKernelGGL((gated_bwd_kernel<IO, V, false, true>), grid, block, 0, stream, a,
                         states, part, g, n);
    else
      hipLaunchKernelGGL((gated_bwd_kernel<IO, V, false, false>), grid, block, 0, stream, a,
                         states, part, g, n);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(gated_reduce_kernel,
                     dim3(static_cast<unsigned>((a.d_inner + 15) / 16), 3), dim3(256), 0, stream,
                     a, part, a.batch * nseg);
  return hipGetLastError();
}

bool pairs(const GatedArgs& a, int64_t es) {
  const void* all[] = {a.x, a.r, a.i, a.z, a.dout, a.dx, a.dr, a.di, a.z ? a.dz : nullptr};
  uintptr_t bits = 0;
  for (const void* q : all) bits |= reinterpret_cast<uintptr_t>(q);
  return a.d_inner % 2 == 0 && bits % (2 * es) == 0;
}

}  // namespace

size_t gated_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, bool bf16, bool given) {
  return static_cast<size_t>(layout(batch, seqlen, d_inner, bf16, given).total);
}

hipError_t launch_gated_bwd(const GatedArgs& a, bool bf16, hipStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  const Layout l = layout(a.batch, a.seqlen, a.d_inner, bf16, a.states != nullptr);
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
  if (bf16)
    return pairs(a, 2) ? launch<BF16, 2>(a, states, part, stream)
                       : launch<BF16, 1>(a, states, part, stream);
  return pairs(a, 4) ? launch<F32, 2>(a, states, part, stream)
                     : launch<F32, 1>(a, states, part, stream);
}

}  // namespace ss
