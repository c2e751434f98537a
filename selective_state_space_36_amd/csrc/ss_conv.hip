// ss_conv.hip -- the causal depthwise convolution, its gradients and its one-token form.
//
// All three stream: each lane owns V channels, holds their k taps in registers and walks steps
// with the last k - 1 inputs in registers, so an input is read once per wave.  Where sequences
// start inside a row, a mask of the starts, the same for the whole wave (a scalar register), says
// which taps would cross one; steps without a start run without a branch.
//
// What bounds it: the forward memory, the backward memory and the VALU alike.  4 x 4096 x 5120
// bfloat16, four taps, packed: forward 336 MB in 64 us (5.2 TB/s), backward 503 MB in 108 us
// (4.7 TB/s, the VALU issuing in nine tenths of the cycles: 36 operations per element) and 5 us for
// the parameters' sums.
// Why these runs: the forward takes a wave's 16 rows and the 3 before them at once, which
// neighbours find in the cache (8 rows: 3 us more).  The backward needs 3 rows on either side of
// its own, so it walks 64 steps with 8 rows in flight (16 to 128 steps and 4 rows: 2 to 20 us more;
// four channels per lane 10 us more, one 45).  Its branches per step cost 20 us before steps
// without a start got a path of their own.
#include "ss_block.h"
#include "ss_gated_math.h"

#include <type_traits>

namespace ss {
namespace {

constexpr int kFwdSteps = 16;  // steps of one wave of the forward
constexpr int kWaves = 4;      // waves of a workgroup, on consecutive runs of steps
constexpr int kStride = 8;     // steps whose rows the backward has in flight

// One lane's taps: w[j][v] for channels c .. c + V - 1, and the bias.
template <int V, int K>
struct Taps {
  float w[K][V], bias[V];
  __device__ __forceinline__ void load(const ConvArgs& p, int64_t c) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][v] = p.weight[(c + v) * K + j];
      bias[v] = p.bias ? p.bias[c + v] : 0.0f;
    }
  }
};

// What lane j needs of the starts at steps t .. t + n - 1 of row b, n < 64 (steps outside the
// sequence have none; without starts the resource is empty and nothing is read).
__device__ __forceinline__ uint8_t starts_at(const ConvArgs& p, int64_t b, int64_t t, int n) {
  const int lane = threadIdx.x & 63;
  const int64_t skip = t < 0 ? -t : 0;             // steps before the sequence
  int64_t rest = p.seqlen - (t + skip);
  rest = rest < 0 || !p.starts ? 0 : rest < n - skip ? rest : n - skip;
  const rsrc_t r = make_buf(p.starts + (rest > 0 ? b * p.seqlen + t + skip : 0),
                            rest > 0 ? static_cast<uint32_t>(rest) : 0);
  // (lanes before the sequence have offsets past every range)
  return __builtin_amdgcn_raw_buffer_load_b8(r, lane - static_cast<int>(skip), 0, 0);
}
// Bit j: a sequence starts at the step of lane j.
__device__ __forceinline__ uint32_t starts_mask(uint8_t at) {
  return static_cast<uint32_t>(__ballot(at != 0));
}

// The tile of this workgroup.  Where rows are not whole cache lines (`near`) the tiles are dealt to
// the XCDs, which take the workgroups in turn, in runs of neighbours: the parts of a line that
// belong to two channel groups then meet in one L2 (training step, in turn / in runs:
// 4 x 4096 x 5121 287 / 227 us, 4 x 4096 x 5122 244 / 208, 3 x 5000 x 2001 float32 176 / 142).
__device__ __forceinline__ uint32_t tile_of(bool near) {
  constexpr uint32_t kXcds = 8;
  const uint32_t x = blockIdx.x % kXcds, all = gridDim.x;
  if (!near) return blockIdx.x;
  return all / kXcds * x + (x < all % kXcds ? x : all % kXcds) + blockIdx.x / kXcds;
}

// Where a wave works: a run of steps of one batch row and 64 V channels.
struct Place {
  int64_t b, t0, c;
  bool active;
};
template <int V>
__device__ __forceinline__ Place place(const ConvArgs& p, int64_t group, int64_t item,
                                       int64_t runs, int64_t run_steps) {
  const int64_t c0 = group * (64 * V) + static_cast<int64_t>(threadIdx.x & 63) * V;
  const bool active = c0 < p.d_inner;
  return Place{item / runs, item % runs * run_steps, active ? c0 : 0, active};
}

// The k - 1 rows before step t0 (t0 is 0 or at least k - 1): of x, or of x_prev, or none.
template <class IO, int V, int K>
__device__ __forceinline__ Rows<IO, V> rows_before(const ConvArgs& p, int64_t b, int64_t t0) {
  const uint32_t bytes = static_cast<uint32_t>((K - 1) * p.d_inner) * sizeof(typename IO::elem);
  if (t0 > 0) return rows_of<IO, V>(p.x, (b * p.seqlen + t0 - (K - 1)) * p.d_inner, bytes);
  return rows_of<IO, V>(p.x_prev, p.x_prev ? b * (K - 1) * p.d_inner : 0, p.x_prev ? bytes : 0);
}

template <class IO, int V, int K, bool SILU, bool PAST>
__global__ __launch_bounds__(64 * kWaves) void conv_fwd_kernel(ConvArgs p, uint32_t groups,
                                                               int64_t runs) {
  using elem = typename IO::elem;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = tile_of(p.d_inner * sizeof(elem) % 128 != 0);
  const int64_t item = static_cast<int64_t>(tile / groups) * kWaves + wave;
  if (item >= p.batch * runs) return;
  const Place at = place<V>(p, tile % groups, item, runs, kFwdSteps);
  const int64_t left = p.seqlen - at.t0;
  const int n = left < kFwdSteps ? static_cast<int>(left) : kFwdSteps;
  const uint32_t row = static_cast<uint32_t>(p.d_inner) * sizeof(elem);
  const uint32_t col = at.active ? static_cast<uint32_t>(at.c) * sizeof(elem) : kOffNone;
  const int64_t first = (at.b * p.seqlen + at.t0) * p.d_inner;
  const auto H = rows_before<IO, V, K>(p, at.b, at.t0);
  const auto X = rows_of<IO, V>(p.x, first, n * row);
  const uint8_t begins = starts_at(p, at.b, at.t0 - (K - 1), kFwdSteps + K - 1);
  typename Lanes<IO, V>::raw x[kFwdSteps + K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) x[j] = H.load(col + j * row);
#pragma unroll
  for (int j = 0; j < kFwdSteps; ++j) x[K - 1 + j] = X.load(col + j * row);
  Taps<V, K> taps;
  taps.load(p, at.c);
  const uint32_t mask = starts_mask(begins);  // bit j: a sequence starts at the row of x[j]
  const auto O = rows_of<IO, V, PAST>(p.out, first, n * row);
  auto step = [&](int j, auto plain) {
    float y[V];
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = taps.bias[v];
#pragma unroll
    for (int q = 0; q < K; ++q) {  // x[j + q] is K - 1 - q steps back
      // a start at one of the steps after that row, up to this one, cuts it off
      const uint32_t between = ((1u << (K - 1 - q)) - 1) << (j + q + 1);
      if (!decltype(plain)::value && (mask & between)) continue;
#pragma unroll
      for (int v = 0; v < V; ++v)
        y[v] = fmaf(taps.w[q][v], Lanes<IO, V>::get(x[j + q], v), y[v]);
    }
    if (SILU) {
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = silu_f(y[v]);
    }
    O.store(y, col + j * row);
  };
  if (mask == 0) {
#pragma unroll
    for (int j = 0; j < kFwdSteps; ++j) step(j, std::true_type{});
  } else {
#pragma unroll
    for (int j = 0; j < kFwdSteps; ++j) step(j, std::false_type{});
  }
}

// One wave walks `steps` steps from t0 and the k - 1 after them (whose g the last dx need; their
// own dx and sums belong to the next wave), kStride rows in flight.  The rows of sums of a
// workgroup's waves are added in LDS into part[workgroup][K + 1][d_inner].
template <class IO, int V, int K, bool SILU, bool PAST>
__global__ __launch_bounds__(64 * kWaves) void conv_bwd_kernel(ConvArgs p, uint32_t groups,
                                                               int64_t runs, int32_t steps,
                                                               float* part) {
  using elem = typename IO::elem;
  using L = Lanes<IO, V>;
  __shared__ float fold[kWaves][(K + 1) * V][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = tile_of(p.d_inner * sizeof(elem) % 128 != 0);
  const int64_t line = tile / groups;
  const int64_t item = line * kWaves + wave;
  const bool some = item < p.batch * runs;
  const Place at = place<V>(p, tile % groups, some ? item : 0, runs, steps);
  const int64_t left = p.seqlen - at.t0;
  const int n = !some ? 0 : left < steps ? static_cast<int>(left) : steps;  // steps of its own
  const int all = n + K - 1;                                                // steps it walks
  const int have = !some ? 0 : left < all ? static_cast<int>(left) : all;   // that exist
  const uint32_t row = static_cast<uint32_t>(p.d_inner) * sizeof(elem);
  const uint32_t col = at.active ? static_cast<uint32_t>(at.c) * sizeof(elem) : kOffNone;
  const int64_t first = (at.b * p.seqlen + at.t0) * p.d_inner;

  float dw[K][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][v] = 0.0f;
  }
  if (some) {
    Taps<V, K> taps;
    taps.load(p, at.c);
    // x and g at the K - 1 steps before the current one and, last, at the current one
    float xw[K][V], gw[K][V];
    {
      const auto H = rows_before<IO, V, K>(p, at.b, at.t0);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const auto raw = H.load(col + j * row);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          xw[j][v] = L::get(raw, v);
          gw[j][v] = 0.0f;
        }
      }
    }
    const bool prev = at.t0 == 0 && p.dx_prev;
    const auto DP = rows_of<IO, V, PAST>(p.dx_prev, prev ? at.b * (K - 1) * p.d_inner : 0,
                                         prev ? (K - 1) * row : 0);
    typename L::raw xn[kStride], gn[kStride];
    // starts at the K - 1 steps before s0, then from s0 on
    uint32_t begins = starts_mask(starts_at(p, at.b, at.t0 - (K - 1), K - 1));
    uint8_t starts = 0;
    // rows are addressed kStride at a time, so that 32-bit offsets reach for any d_inner
    auto fetch = [&](int s0) {
      const int more = have - s0 < 0 ? 0 : have - s0 < kStride ? have - s0 : kStride;
      const int64_t f = more ? first + s0 * p.d_inner : 0;
      const auto X = rows_of<IO, V, PAST>(p.x, f, more * row);
      const auto G = rows_of<IO, V, PAST>(p.dout, f, more * row);
#pragma unroll
      for (int j = 0; j < kStride; ++j) {
        xn[j] = X.load(col + j * row);
        gn[j] = G.load(col + j * row);
      }
      starts = starts_at(p, at.b, at.t0 + s0, kStride);
    };
    fetch(0);
    for (int s0 = 0; s0 < all; s0 += kStride) {
      typename L::raw xr[kStride], gr[kStride];
#pragma unroll
      for (int j = 0; j < kStride; ++j) {
        xr[j] = xn[j];
        gr[j] = gn[j];
      }
      begins |= starts_mask(starts) << (K - 1);  // bit j + K - 1: a sequence starts at step s0 + j
      const uint32_t now = begins;
      // dx trails by K - 1 steps
      static_assert(kStride >= K, "the first rows hold a whole window");
      const int skip = s0 ? 0 : K - 1, r0 = s0 ? s0 - (K - 1) : 0;
      const int rest = n - r0 < 0 ? 0 : n - r0 < kStride ? n - r0 : kStride;
      const auto DX = rows_of<IO, V, PAST>(p.dx, first + (rest ? r0 * p.d_inner : 0), rest * row);
      if (s0 + kStride < all) fetch(s0 + kStride);
      // Step s0 + j.  PLAIN: all of the kStride steps are the wave's own and no sequence starts
      // among them or in the window, so that nothing in them branches.
      auto step = [&](int j, auto plain) {
        constexpr bool kPlain = decltype(plain)::value;
        const int s = s0 + j;
        float g[V], pre[V], dx[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          xw[K - 1][v] = L::get(xr[j], v);
          g[v] = L::get(gr[j], v);
          pre[v] = taps.bias[v];
        }
        // whether a start cuts tap q (the row K - 1 - q steps back) off from this step, and this
        // step's g (q steps after it) from the step K - 1 back
        auto tap_cut = [&](int q) { return now & (((1u << (K - 1 - q)) - 1) << (j + q + 1)); };
        auto dx_cut = [&](int q) { return now & (((1u << q) - 1) << (j + 1)); };
#pragma unroll
        for (int q = 0; q < K; ++q) {
          if (!kPlain && tap_cut(q)) continue;
#pragma unroll
          for (int v = 0; v < V; ++v) pre[v] = fmaf(taps.w[q][v], xw[q][v], pre[v]);
        }
        if (SILU) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float sg = sigmoid_f(pre[v]);
            // silu' = sg (1 + pre (1 - sg))
            g[v] *= fmaf(sg, fmaf(-pre[v], sg, pre[v]), sg);
          }
        }
        if (!kPlain && s >= have) {  // past the end: no gradient, whatever silu' gave
#pragma unroll
          for (int v = 0; v < V; ++v) g[v] = 0.0f;
        }
        if (kPlain || s < n) {
#pragma unroll
          for (int v = 0; v < V; ++v) db[v] += g[v];
#pragma unroll
          for (int q = 0; q < K; ++q) {
            if (!kPlain && tap_cut(q)) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) dw[q][v] = fmaf(g[v], xw[q][v], dw[q][v]);
          }
        }
        // the step K - 1 back now has every g it takes part in: gw[q] is g at q steps after it
#pragma unroll
        for (int v = 0; v < V; ++v) {
          gw[K - 1][v] = g[v];
          dx[v] = 0.0f;
        }
#pragma unroll
        for (int q = 0; q < K; ++q) {
          if (!kPlain && dx_cut(q)) continue;
#pragma unroll
          for (int v = 0; v < V; ++v) dx[v] = fmaf(taps.w[K - 1 - q][v], gw[q][v], dx[v]);
        }
        if (j >= K - 1 || s0)
          DX.store(dx, col + (j - skip) * row);
        else if (prev)
          DP.store(dx, col + s * row);
#pragma unroll
        for (int q = 0; q + 1 < K; ++q) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            xw[q][v] = xw[q + 1][v];
            gw[q][v] = gw[q + 1][v];
          }
        }
      };
      if (s0 + kStride <= n && now == 0) {
#pragma unroll
        for (int j = 0; j < kStride; ++j) step(j, std::true_type{});
      } else {
#pragma unroll
        for (int j = 0; j < kStride; ++j) {
          if (s0 + j < all) step(j, std::false_type{});
        }
      }
      begins = now >> kStride;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int q = 0; q < K; ++q) fold[wave][q * V + v][lane] = dw[q][v];
    fold[wave][K * V + v][lane] = db[v];
  }
  __syncthreads();
  if (!at.active) return;
  for (int q = wave; q <= K; q += kWaves) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float s = fold[0][q * V + v][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += fold[w][q * V + v][lane];
      part[(line * (K + 1) + q) * p.d_inner + at.c + v] = s;
    }
  }
}

// One token: V channels of one batch row per thread.
template <class IO, int V, int K>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs p, int64_t lanes) {
  using elem = typename IO::elem;
  using raw = typename Lanes<IO, V>::raw;
  const int64_t id = blockIdx.x * 256ll + threadIdx.x;
  if (id >= p.batch * lanes) return;
  const int64_t b = id / lanes, c = id % lanes * V;
  raw* out = reinterpret_cast<raw*>(static_cast<elem*>(p.out) + b * p.d_inner + c);
  raw x[K];
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    x[j] = *reinterpret_cast<const raw*>(static_cast<const elem*>(p.conv_state) +
                                         (b * (K - 1) + j) * p.d_inner + c);
  x[K - 1] = *reinterpret_cast<const raw*>(static_cast<const elem*>(p.x) + b * p.d_inner + c);
  Taps<V, K> taps;
  taps.load(p, c);
  float y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    y[v] = taps.bias[v];
#pragma unroll
    for (int j = 0; j < K; ++j) y[v] = fmaf(taps.w[j][v], Lanes<IO, V>::get(x[j], v), y[v]);
    if (p.silu) y[v] = silu_f(y[v]);
  }
  *out = Lanes<IO, V>::put(y);
#pragma unroll
  for (int j = 0; j + 1 < K; ++j)
    *reinterpret_cast<raw*>(static_cast<elem*>(p.conv_state) + (b * (K - 1) + j) * p.d_inner +
                            c) = x[j + 1];
}

// Steps per wave of the backward: long runs walk the k - 1 steps after them the fewest times, as
// long as there are enough of them for one per SIMD (1024).
int64_t bwd_steps(int64_t batch, int64_t seqlen, int64_t d_inner) {
  const int64_t runs = (seqlen + 63) / 64, groups = (d_inner + 127) / 128;
  return batch * runs * groups >= 1024 ? 64 : 16;
}
int64_t lines_of(int64_t batch, int64_t seqlen, int64_t steps) {
  return (batch * ((seqlen + steps - 1) / steps) + kWaves - 1) / kWaves;
}

template <class F>
void with_width(int32_t k, F f) {
  using std::integral_constant;
  if (k == 1) f(integral_constant<int, 1>{});
  else if (k == 2) f(integral_constant<int, 2>{});
  else if (k == 3) f(integral_constant<int, 3>{});
  else f(integral_constant<int, 4>{});
}

template <class IO, int V>
hipError_t launch_fwd(const ConvArgs& a, hipStream_t stream) {
  const int64_t groups = (a.d_inner + 64 * V - 1) / (64 * V);
  const int64_t runs = (a.seqlen + kFwdSteps - 1) / kFwdSteps;
  const dim3 grid(static_cast<unsigned>((a.batch * runs + kWaves - 1) / kWaves * groups));
  const dim3 block(64 * kWaves);
  const uint32_t g = static_cast<uint32_t>(groups);
  const int64_t bytes = a.batch * a.seqlen * a.d_inner * sizeof(typename IO::elem);
  with_width(a.k, [&](auto k) {
    auto go = [&](auto silu, auto past) {
      hipLaunchKernelGGL((conv_fwd_kernel<IO, V, k, silu, past>), grid, block, 0, stream, a, g,
                         runs);
    };
    with_bools(go, a.silu, passes_cache(2 * bytes, a.d_inner * sizeof(typename IO::elem)));
  });
  return hipGetLastError();
}

template <class IO, int V>
hipError_t launch_bwd(const ConvArgs& a, hipStream_t stream) {
  const int64_t groups = (a.d_inner + 64 * V - 1) / (64 * V);
  const int32_t steps = static_cast<int32_t>(bwd_steps(a.batch, a.seqlen, a.d_inner));
  const int64_t runs = (a.seqlen + steps - 1) / steps;
  const int64_t lines = lines_of(a.batch, a.seqlen, steps);
  const dim3 grid(static_cast<unsigned>(lines * groups)), block(64 * kWaves);
  const uint32_t g = static_cast<uint32_t>(groups);
  const int64_t bytes = a.batch * a.seqlen * a.d_inner * sizeof(typename IO::elem);
  float* part = static_cast<float*>(a.workspace);
  with_width(a.k, [&](auto k) {
    auto go = [&](auto silu, auto past) {
      hipLaunchKernelGGL((conv_bwd_kernel<IO, V, k, silu, past>), grid, block, 0, stream, a, g,
                         runs, steps, part);
    };
    with_bools(go, a.silu, passes_cache(3 * bytes, a.d_inner * sizeof(typename IO::elem)));
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  ColumnSums c{};
  c.lines = lines;
  c.stride = (a.k + 1) * a.d_inner;
  c.cols = a.d_inner;
  for (int q = 0; q < a.k; ++q) c.add(part + q * a.d_inner, a.dweight + q, a.k);
  c.add(part + a.k * a.d_inner, a.dbias, 1);
  return launch_column_sums(c, stream);
}

template <class IO, int V>
hipError_t launch_step(const ConvArgs& a, hipStream_t stream) {
  const int64_t lanes = a.d_inner / V;
  const dim3 grid(static_cast<unsigned>((a.batch * lanes + 255) / 256));
  with_width(a.k, [&](auto k) {
    hipLaunchKernelGGL((conv_step_kernel<IO, V, k>), grid, dim3(256), 0, stream, a, lanes);
  });
  return hipGetLastError();
}

// Whether v channels per lane fit: whole groups, and every io pointer aligned to one.
template <class IO>
bool lanes_of(const ConvArgs& a, int v) {
  const void* all[] = {a.x, a.x_prev, a.out, a.conv_state, a.dout, a.dx, a.dx_prev};
  uintptr_t bits = 0;
  for (const void* q : all) bits |= reinterpret_cast<uintptr_t>(q);
  return a.d_inner % v == 0 && bits % (v * sizeof(typename IO::elem)) == 0;
}

}  // namespace

size_t conv_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, int32_t k) {
  const int64_t lines = lines_of(batch, seqlen, bwd_steps(batch, seqlen, d_inner));
  return static_cast<size_t>(lines * (k + 1) * d_inner) * sizeof(float);
}

hipError_t launch_conv_fwd(const ConvArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) {
    if (lanes_of<BF16>(a, 4)) return launch_fwd<BF16, 4>(a, stream);
    return lanes_of<BF16>(a, 2) ? launch_fwd<BF16, 2>(a, stream) : launch_fwd<BF16, 1>(a, stream);
  }
  return lanes_of<F32>(a, 2) ? launch_fwd<F32, 2>(a, stream) : launch_fwd<F32, 1>(a, stream);
}

hipError_t launch_conv_bwd(const ConvArgs& a, bool bf16, hipStream_t stream) {
  if (bf16)
    return lanes_of<BF16>(a, 2) ? launch_bwd<BF16, 2>(a, stream) : launch_bwd<BF16, 1>(a, stream);
  return lanes_of<F32>(a, 2) ? launch_bwd<F32, 2>(a, stream) : launch_bwd<F32, 1>(a, stream);
}

hipError_t launch_conv_step(const ConvArgs& a, bool bf16, hipStream_t stream) {
  if (bf16)
    return lanes_of<BF16>(a, 4) ? launch_step<BF16, 4>(a, stream)
                                : launch_step<BF16, 1>(a, stream);
  return lanes_of<F32>(a, 4) ? launch_step<F32, 4>(a, stream) : launch_step<F32, 1>(a, stream);
}

}  // namespace ss
