// ss_gated_fwd.hip -- the gated linear recurrence over a whole sequence.
//
// One workgroup per tile of kWaves x kSteps steps by 64 V channels; wave w owns kSteps consecutive
// steps.  Each lane loads its steps of its V channels at once, forms decay and input in registers,
// and reduces them to a Piece; the waves' pieces meet in LDS, the tile's goes to the chain
// (ss_gated_chain.h), and with the state before its first step every wave runs its steps again
// from the registers and stores.  Inputs are read once and outputs written once.
#include "ss_block.h"
#include "ss_gated_chain.h"

namespace ss {
namespace {

constexpr int kSteps = 8;
constexpr int kWaves = 8;
constexpr int kTile = kSteps * kWaves;

template <class IO, int V, bool GATE, bool PACKED>
__global__ __launch_bounds__(64 * kWaves) void gated_fwd_kernel(GatedArgs p, int32_t groups,
                                                                int32_t nseg) {
  using elem = typename IO::elem;
  using L = Lanes<IO, V>;
  __shared__ Piece pieces[kWaves][V][64];
  __shared__ slot_t look[kWaves * V * 64];
  __shared__ uint32_t drawn;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const uint32_t chains = static_cast<uint32_t>(p.batch) * groups;
  uint32_t* counter = static_cast<uint32_t*>(p.workspace);
  const uint32_t tile = nseg > 1 ? draw_tile(counter, &drawn) : blockIdx.x;
  const uint32_t seg = tile / chains, chain = tile % chains;
  const int64_t b = chain / groups;
  const int64_t c0 = static_cast<int64_t>(chain % groups) * (64 * V) + lane * V;
  const bool active = c0 < p.d_inner;
  const int64_t c = active ? c0 : 0;
  const int64_t t0 = static_cast<int64_t>(seg) * kTile + wave * kSteps;
  const int64_t row0 = b * p.seqlen;
  // the wave's rows: kSteps of them, or what is left of the sequence (none past its end)
  const int64_t left = p.seqlen - t0;
  const int n = left < 0 ? 0 : left < kSteps ? static_cast<int>(left) : kSteps;
  const int64_t first = (row0 + t0) * p.d_inner;
  const uint32_t row = static_cast<uint32_t>(p.d_inner) * sizeof(elem);
  const uint32_t col = active ? static_cast<uint32_t>(c) * sizeof(elem) : kOffNone;
  auto rows = [&](const void* base) { return rows_of<IO, V>(base, n ? first : 0, n * row); };
  typename L::raw xr[kSteps], rr[kSteps], ir[kSteps], zr[kSteps];
  {
    const Rows<IO, V> R = rows(p.r), I = rows(p.i), X = rows(p.x);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      rr[j] = R.load(col + j * row);
      ir[j] = I.load(col + j * row);
      xr[j] = X.load(col + j * row);
    }
  }
  uint32_t fresh = 0;  // bit j: a sequence starts at step j
  if (PACKED) fresh = static_cast<uint32_t>(__ballot(lane < n && p.starts[row0 + t0 + lane]));
  float A[V], rb[V], ib[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = p.A[c + v];
    rb[v] = p.r_bias ? p.r_bias[c + v] : 0.0f;
    ib[v] = p.i_bias ? p.i_bias[c + v] : 0.0f;
  }

  float a[kSteps][V], in[kSteps][V];
  Piece piece[V];
#pragma unroll
  for (int v = 0; v < V; ++v) piece[v] = Piece{1.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const bool beyond = j >= n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float rg = sigmoid_f(L::get(rr[j], v) + rb[v]);
      const float ig = sigmoid_f(L::get(ir[j], v) + ib[v]);
      const Decay k = decay_f(A[v] * rg);
      a[j][v] = beyond ? 1.0f : fmaxf(k.a, kTinyDecay);
      in[j][v] = beyond ? 0.0f : k.s * ig * L::get(xr[j], v);
      const bool cut = PACKED && (fresh >> j & 1);
      piece[v].H = cut ? in[j][v] : fmaf(a[j][v], piece[v].H, in[j][v]);
      piece[v].P = fmaxf(piece[v].P * a[j][v], kTinyDecay);
    }
  }
  if (PACKED && fresh) {
#pragma unroll
    for (int v = 0; v < V; ++v) piece[v].P = 0.0f;
  }
  if (GATE) {
    const Rows<IO, V> Z = rows(p.z);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) zr[j] = Z.load(col + j * row);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) pieces[wave][v][lane] = piece[v];
  __syncthreads();

  float h[V];
  if (nseg > 1) {
    Piece whole[V];
    slot_t* slots = reinterpret_cast<slot_t*>(static_cast<char*>(p.workspace) + kChainHead) +
                    static_cast<int64_t>(chain) * (64 * V) + lane * V;
    const int64_t stride = static_cast<int64_t>(chains) * (64 * V);
    if (wave == 0 && static_cast<int32_t>(seg) + 1 < nseg) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        whole[v] = pieces[0][v][lane];
        for (int k = 1; k < waves; ++k) whole[v] = then(whole[v], pieces[k][v][lane]);
        if (seg) publish(slots + seg * stride + v, whole[v]);
      }
    }
    if (seg) {
      state_before<V>(slots, stride, seg, look, h);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = p.h0 ? p.h0[b * p.d_inner + c + v] : 0.0f;
    }
    if (wave == 0 && static_cast<int32_t>(seg) + 1 < nseg) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        publish(slots + seg * stride + v, Piece{0.0f, advance(whole[v], h[v])});
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = p.h0 ? p.h0[b * p.d_inner + c + v] : 0.0f;
  }
  for (int k = 0; k < wave; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = advance(pieces[k][v][lane], h[v]);
  }

  const Rows<IO, V> O = rows(p.out);
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    float y[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool cut = PACKED && (fresh >> j & 1);
      h[v] = cut ? in[j][v] : fmaf(a[j][v], h[v], in[j][v]);
      y[v] = GATE ? h[v] * silu_f(L::get(zr[j], v)) : h[v];
    }
    if (p.out) O.store(y, col + j * row);
  }
  // The wave that holds the last step of a chunk or of the sequence (its steps past the end left
  // the state as it was).
  static_assert(SS_GATED_CHUNK % kSteps == 0, "a chunk ends with a wave's last step");
  if (n > 0 && active) {
    if (p.states && (left <= kSteps || (t0 + kSteps) % SS_GATED_CHUNK == 0)) {
      float* s = p.states + (b * p.n_chunks + t0 / SS_GATED_CHUNK) * p.d_inner + c;
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = h[v];
    }
    if (p.h_last && left <= kSteps) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.h_last[b * p.d_inner + c + v] = h[v];
    }
  }
}

int64_t segments_of(int64_t seqlen) { return (seqlen + kTile - 1) / kTile; }

template <class IO, int V>
hipError_t launch(const GatedArgs& a, hipStream_t stream) {
  const int64_t groups = (a.d_inner + 64 * V - 1) / (64 * V);
  const int64_t nseg = segments_of(a.seqlen);
  const int64_t tiles = a.batch * groups * nseg;
  if (tiles > 0x7fffffff) return hipErrorInvalidValue;
  if (nseg > 1) {
    const int64_t bytes = kChainHead + tiles * (64 * V) * static_cast<int64_t>(sizeof(slot_t));
    const hipError_t e = launch_zero(static_cast<float*>(a.workspace), bytes / 4, stream);
    if (e != hipSuccess) return e;
  }
  // a sequence shorter than a tile needs fewer waves
  const int waves = nseg > 1 ? kWaves : static_cast<int>((a.seqlen + kSteps - 1) / kSteps);
  const dim3 grid(static_cast<unsigned>(tiles)), block(64 * waves);
  const int32_t g = static_cast<int32_t>(groups), n = static_cast<int32_t>(nseg);
  if (a.z) {
    if (a.starts)
      hipLaunchKernelGGL((gated_fwd_kernel<IO, V, true, true>), grid, block, 0, stream, a, g, n);
    else
      hipLaunchKernelGGL((gated_fwd_kernel<IO, V, true, false>), grid, block, 0, stream, a, g, n);
  } else {
    if (a.starts)
      hipLaunchKernelGGL((gated_fwd_kernel<IO, V, false, true>), grid, block, 0, stream, a, g, n);
    else
      hipLaunchKernelGGL((gated_fwd_kernel<IO, V, false, false>), grid, block, 0, stream, a, g,
                         n);
  }
  return hipGetLastError();
}

// Two channels per lane need rows and pointers aligned to both.
bool pairs(const GatedArgs& a, int64_t es) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.r) |
                        reinterpret_cast<uintptr_t>(a.i) | reinterpret_cast<uintptr_t>(a.z) |
                        reinterpret_cast<uintptr_t>(a.out);
  return a.d_inner % 2 == 0 && all % (2 * es) == 0;
}

}  // namespace

size_t gated_fwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, bool) {
  const int64_t nseg = segments_of(seqlen);
  if (nseg <= 1) return 0;
  const int64_t width = (d_inner + 127) / 128 * 128;  // a whole number of groups of 64 or 128
  return static_cast<size_t>(kChainHead + batch * nseg * width *
                             static_cast<int64_t>(sizeof(slot_t)));
}

hipError_t launch_gated_fwd(const GatedArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) return pairs(a, 2) ? launch<BF16, 2>(a, stream) : launch<BF16, 1>(a, stream);
  return pairs(a, 4) ? launch<F32, 2>(a, stream) : launch<F32, 1>(a, stream);
}

}  // namespace ss
