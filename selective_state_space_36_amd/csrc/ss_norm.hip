// ss_norm.hip -- layer norm over the last axis with the residual add, and its gradients.
//
// A row lies in the registers of TPR threads (64, 256 or 1024), K groups of V consecutive columns
// each, so it is read once: the mean, then the squared differences from it, then the output all
// come from the same registers.  Sums run over the lanes of a wave by DPP, over the waves through
// LDS.  Rows too wide for that (over 16384 columns, 12288 in the backward, or 8192 that are not
// groups of four) are read again for each pass by the wide kernels.
//
// What bounds it: memory.  16384 x 2560 bfloat16 with the residual stream: forward 503 MB in 97 us
// (5.2 TB/s), backward 671 MB in 106 us and 5 us for the parameters' sums (6.3 TB/s, some of it
// from the 256 MB cache); a copy of 1 GB reaches 5.0 TB/s.  The backward asks for a row's successor
// before it sums the row.  The wide kernels are bound by their passes, of single columns a lane:
// 2048 x 32768, forward 403 MB in 400 us, backward 537 MB in 364 us.
#include "ss_block.h"
#include "ss_rows.h"

#include <type_traits>

namespace ss {
namespace {

// Sum over the wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  v += row_ror<1>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Sums of N values over the TPR threads of a row, the same in every thread.  `lds` holds N rows
// of 16 floats; `phase` alternates between two of them, so that one barrier per sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* lds, int phase) {
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] = wave_sum(v[q]);
  if constexpr (TPR > 64) {
    constexpr int kW = TPR / 64;
    float* at = lds + (phase & 1) * N * 16;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int q = 0; q < N; ++q) at[q * 16 + (threadIdx.x >> 6)] = v[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < N; ++q) {
      float s = at[q * 16];
#pragma unroll
      for (int w = 1; w < kW; ++w) s += at[q * 16 + w];
      v[q] = s;
    }
  }
}

template <int TPR>
constexpr int kBlock = TPR < 256 ? 256 : TPR;  // threads of a workgroup

template <class IO, int V, int TPR, int K, bool PAST>
__global__ __launch_bounds__(kBlock<TPR>) void norm_fwd_kernel(NormArgs p) {
  __shared__ float lds[2 * 16];
  constexpr int kRows = kBlock<TPR> / TPR;
  const int tid = threadIdx.x % TPR;
  const int sub = kRows > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0;
  const uint32_t dim = static_cast<uint32_t>(p.dim);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub; row < p.rows; row += stride) {
    const int64_t at = row * p.dim;
    const auto X = rows_of<IO, V, PAST>(p.x, at, dim * sizeof(typename IO::elem));
    const auto W = rows_of<F32, V>(p.weight, 0, p.weight ? dim * 4 : 0);
    const auto B = rows_of<F32, V>(p.bias, 0, p.bias ? dim * 4 : 0);
    typename Lanes<IO, V>::raw xr[K];
    typename Lanes<F32, V>::raw rr[K], wr[K], br[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t col = (k * TPR + tid) * V;
      xr[k] = X.load(col * sizeof(typename IO::elem));
    }
    if (p.residual) {
      const auto R = rows_of<F32, V, PAST>(p.residual, at, dim * 4);
#pragma unroll
      for (int k = 0; k < K; ++k) rr[k] = R.load((k * TPR + tid) * V * 4);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      wr[k] = W.load((k * TPR + tid) * V * 4);
      br[k] = B.load((k * TPR + tid) * V * 4);
    }
    float s[K][V], sum[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[k][v] = Lanes<IO, V>::get(xr[k], v);
        if (p.residual) s[k][v] += Lanes<F32, V>::get(rr[k], v);
        sum[0] += s[k][v];
      }
    }
    if (p.sum) {
      const auto S = rows_of<F32, V>(p.sum, at, dim * 4);
#pragma unroll
      for (int k = 0; k < K; ++k) S.store(s[k], (k * TPR + tid) * V * 4);
    }
    const float n = static_cast<float>(p.dim);
    row_sums<TPR>(sum, lds, 0);
    const float mu = sum[0] / n;
    float sq[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = (k * TPR + tid) * V < dim;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[k][v] -= mu;
        const float c = in ? s[k][v] : 0.0f;
        sq[0] = fmaf(c, c, sq[0]);
      }
    }
    row_sums<TPR>(sq, lds, 1);
    const float rstd = 1.0f / __builtin_sqrtf(sq[0] / n + p.eps);
    const auto O = rows_of<IO, V>(p.out, at, dim * sizeof(typename IO::elem));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float w = p.weight ? Lanes<F32, V>::get(wr[k], v) : 1.0f;
        y[v] = fmaf(s[k][v] * rstd, w, Lanes<F32, V>::get(br[k], v));
      }
      O.store(y, (k * TPR + tid) * V * sizeof(typename IO::elem));
    }
    if (tid == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

// Each row group of the launch walks the rows with the launch's stride and adds dweight and dbias
// in its registers; part[strand][2][dim] takes one line per workgroup.
template <class IO, class S, int V, int TPR, int K, bool PAST>
__global__ __launch_bounds__(kBlock<TPR>) void norm_bwd_kernel(NormArgs p, float* part) {
  constexpr int kRows = kBlock<TPR> / TPR;
  __shared__ float lds[4 * 16];
  __shared__ float fold[kRows > 1 ? kRows * 2 * V * K * TPR : 1];
  const int tid = threadIdx.x % TPR;
  const int sub = kRows > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0;
  const uint32_t dim = static_cast<uint32_t>(p.dim);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  const float inv = 1.0f / static_cast<float>(p.dim);
  const auto W = rows_of<F32, V>(p.weight, 0, p.weight ? dim * 4 : 0);
  float w[K][V], dw[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const auto wr = W.load((k * TPR + tid) * V * 4);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[k][v] = p.weight ? Lanes<F32, V>::get(wr, v) : 1.0f;
      dw[k][v] = db[k][v] = 0.0f;
    }
  }
  typename Lanes<IO, V>::raw gr[K];
  typename Lanes<S, V>::raw sr[K];
  typename Lanes<F32, V>::raw ur[K];
  float mu = 0.0f, rstd = 0.0f;
  // A row past the last one reads as zeros, without an access (empty resources).
  auto fetch = [&](int64_t row) {
    const bool in = row < p.rows;
    const int64_t at = in ? row * p.dim : 0;
    const auto G = rows_of<IO, V, PAST>(p.dout, at, in ? dim * sizeof(typename IO::elem) : 0);
    const auto X = rows_of<S, V, PAST>(p.x, at, in ? dim * sizeof(typename S::elem) : 0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      gr[k] = G.load((k * TPR + tid) * V * sizeof(typename IO::elem));
      sr[k] = X.load((k * TPR + tid) * V * sizeof(typename S::elem));
    }
    if (p.dsum) {
      const auto U = rows_of<F32, V, PAST>(p.dsum, at, in ? dim * 4 : 0);
#pragma unroll
      for (int k = 0; k < K; ++k) ur[k] = U.load((k * TPR + tid) * V * 4);
    }
    mu = in ? p.mean_in[row] : 0.0f;
    rstd = in ? p.rstd_in[row] : 0.0f;
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub;
  fetch(row);
  int phase = 0;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < p.rows;
       first += stride, row += stride, ++phase) {
    float xh[K][V], g[K][V], u[K][V], sums[2] = {0.0f, 0.0f};
    const float rs = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = (k * TPR + tid) * V < dim;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float dy = Lanes<IO, V>::get(gr[k], v);
        xh[k][v] = in ? (Lanes<S, V>::get(sr[k], v) - mu) * rs : 0.0f;
        g[k][v] = dy * w[k][v];
        dw[k][v] = fmaf(dy, xh[k][v], dw[k][v]);
        db[k][v] += dy;
        sums[0] += g[k][v];
        sums[1] = fmaf(g[k][v], xh[k][v], sums[1]);
        u[k][v] = p.dsum ? Lanes<F32, V>::get(ur[k], v) : 0.0f;
      }
    }
    fetch(row + stride);  // in flight over the sums and the stores
    row_sums<TPR>(sums, lds, phase);
    const float c1 = sums[0] * inv, c2 = sums[1] * inv;
    const bool live = row < p.rows;
    const int64_t at = live ? row * p.dim : 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) u[k][v] = fmaf(rs, g[k][v] - c1 - xh[k][v] * c2, u[k][v]);
    }
    if (p.dx) {
      const auto O = rows_of<IO, V>(p.dx, at, live ? dim * sizeof(typename IO::elem) : 0);
#pragma unroll
      for (int k = 0; k < K; ++k) O.store(u[k], (k * TPR + tid) * V * sizeof(typename IO::elem));
    }
    if (p.dresidual) {
      const auto O = rows_of<F32, V>(p.dresidual, at, live ? dim * 4 : 0);
#pragma unroll
      for (int k = 0; k < K; ++k) O.store(u[k], (k * TPR + tid) * V * 4);
    }
  }
  if (!part) return;
  if constexpr (kRows > 1) {  // the row groups' sums into the first one's, in order
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        fold[((sub * 2 * K + k) * V + v) * TPR + tid] = dw[k][v];
        fold[((sub * 2 * K + K + k) * V + v) * TPR + tid] = db[k][v];
      }
    }
    __syncthreads();
    if (sub) return;
    for (int r = 1; r < kRows; ++r) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          dw[k][v] += fold[((r * 2 * K + k) * V + v) * TPR + tid];
          db[k][v] += fold[((r * 2 * K + K + k) * V + v) * TPR + tid];
        }
      }
    }
  }
  const int64_t line = static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
  const auto PW = rows_of<F32, V>(part, line, dim * 4);
  const auto PB = rows_of<F32, V>(part, line + p.dim, dim * 4);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    PW.store(dw[k], (k * TPR + tid) * V * 4);
    PB.store(db[k], (k * TPR + tid) * V * 4);
  }
}

// ------------------------------------------------------------------------------------- wide rows

constexpr int kWide = 1024;

template <class IO>
__global__ __launch_bounds__(kWide) void norm_fwd_wide_kernel(NormArgs p) {
  using elem = typename IO::elem;
  __shared__ float lds[2 * 16];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at = row * p.dim;
    auto value = [&](int64_t c) {
      const float x = IO::load(static_cast<const elem*>(p.x), at + c);
      return p.residual ? x + p.residual[at + c] : x;
    };
    const float n = static_cast<float>(p.dim);
    float s[1] = {0.0f}, sq[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < p.dim; c += kWide) s[0] += value(c);
    row_sums<kWide>(s, lds, 0);
    const float mu = s[0] / n;
    for (int64_t c = threadIdx.x; c < p.dim; c += kWide) {
      const float t = value(c) - mu;
      sq[0] = fmaf(t, t, sq[0]);
    }
    row_sums<kWide>(sq, lds, 1);
    const float rstd = 1.0f / __builtin_sqrtf(sq[0] / n + p.eps);
    for (int64_t c = threadIdx.x; c < p.dim; c += kWide) {
      const float t = value(c);
      const float w = p.weight ? p.weight[c] : 1.0f, b = p.bias ? p.bias[c] : 0.0f;
      static_cast<elem*>(p.out)[at + c] = IO::from_float(fmaf((t - mu) * rstd, w, b));
      if (p.sum) p.sum[at + c] = t;
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

template <class IO, class S>
__global__ __launch_bounds__(kWide) void norm_bwd_wide_kernel(NormArgs p) {
  using elem = typename IO::elem;
  __shared__ float lds[4 * 16];
  int phase = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++phase) {
    const int64_t at = row * p.dim;
    const float mu = p.mean_in[row], rstd = p.rstd_in[row];
    const auto* sp = static_cast<const typename S::elem*>(p.x);
    auto hat = [&](int64_t c) { return (S::load(sp, at + c) - mu) * rstd; };
    auto grad = [&](int64_t c) {
      return IO::load(static_cast<const elem*>(p.dout), at + c) * (p.weight ? p.weight[c] : 1.0f);
    };
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < p.dim; c += kWide) {
      const float g = grad(c);
      s[0] += g;
      s[1] = fmaf(g, hat(c), s[1]);
    }
    row_sums<kWide>(s, lds, phase);
    const float inv = 1.0f / static_cast<float>(p.dim);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    for (int64_t c = threadIdx.x; c < p.dim; c += kWide) {
      const float ds = fmaf(rstd, grad(c) - c1 - hat(c) * c2, p.dsum ? p.dsum[at + c] : 0.0f);
      if (p.dx) static_cast<elem*>(p.dx)[at + c] = IO::from_float(ds);
      if (p.dresidual) p.dresidual[at + c] = ds;
    }
  }
}

// dweight and dbias of wide rows: one thread per column and strand of rows.
template <class IO, class S>
__global__ __launch_bounds__(256) void norm_param_wide_kernel(NormArgs p, float* part) {
  using elem = typename IO::elem;
  const int64_t c = blockIdx.x * 256ll + threadIdx.x;
  if (c >= p.dim) return;
  const auto* sp = static_cast<const typename S::elem*>(p.x);
  float w = 0.0f, b = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float dy = IO::load(static_cast<const elem*>(p.dout), row * p.dim + c);
    w = fmaf(dy, (S::load(sp, row * p.dim + c) - p.mean_in[row]) * p.rstd_in[row], w);
    b += dy;
  }
  part[(2 * static_cast<int64_t>(blockIdx.y)) * p.dim + c] = w;
  part[(2 * static_cast<int64_t>(blockIdx.y) + 1) * p.dim + c] = b;
}

// --------------------------------------------------------------------------------------- dispatch

// Threads per row: the fewest that hold it in registers, 0 for a wide row.  (At most 8 single
// columns per thread, so more threads, took 342 against 244 us for a training step at 16384 x 2561,
// 162 against 95 at 8000 x 2049; 226 against 198 at 8000 x 4093, float32 239 against 248.)
//
// 1024 threads have 128 registers each and hold up to `rounds` groups of four columns, or 8 single
// ones, per thread.  Measured in registers / by the wide kernels, us, bfloat16 with a residual and
// float32 without: forward 4096 x 16384 154 / 403 and 104 / 221, singles 4096 x 8191 97 / 204 and
// 4096 x 4101 58 / 97 and 29 / 47.  The backward keeps nine values per column.  In a third round it
// spills 8 to 21 registers, which still pays (4096 x 8196 153 / 203, 4096 x 12288 192 / 270 and
// 164 / 255; not where everything lies in the cache, 512 x 12288 58 / 35); in a fourth 50 to 62,
// which does not (4096 x 12292 409 / 284, 4096 x 16384 442 / 346 and 445 / 327, 512 x 12292 86 /
// 37; one to 64 rows of 16384, which launches bound, 18 to 25 / 19 to 27).
constexpr int kRoundsFwd = 4, kRoundsBwd = 3;
int threads_per_row(int64_t dim, bool quads, int rounds) {
  return dim <= 64 * 16 ? 64
         : dim <= 256 * 16 ? 256
         : dim <= 1024 * (quads ? 4 * rounds : 8) ? 1024
                                                  : 0;
}

// Lines of partial sums, and with them workgroups of the backward: two per CU fill the card as the
// registers let them, and more lines are more traffic (16384 x 2560: 512 lines 225.7, 768 229.7,
// 1024 233.4, 1536 235.9 us for forward and backward).
constexpr int64_t kStrands = 512;
int64_t strands_of(int64_t rows, int rows_per_group) {
  const int64_t n = (rows + rows_per_group - 1) / rows_per_group;
  return n < kStrands ? n : kStrands;
}

// A workgroup per group of rows, up to `most` (a launch counts its threads in 32 bits); then they
// loop.
unsigned blocks_of(int64_t rows, int64_t rows_per_group, int64_t most) {
  const int64_t n = (rows + rows_per_group - 1) / rows_per_group;
  return static_cast<unsigned>(n < most ? n : most);
}

// Single columns always go through the caches: a line is asked for by several loads of a wave's
// (16384 x 2561 float32, past them 329 us, through 304; 8000 x 6142 333 / 321).
template <int V, class F>
void with_past(F f, bool past) {
  if constexpr (V == 4) {
    if (past) return f(std::true_type{});
  }
  f(std::false_type{});
}

template <class IO, int V, int TPR, int K>
void fwd(const NormArgs& a, hipStream_t stream) {
  constexpr int kRows = kBlock<TPR> / TPR;
  const dim3 grid(blocks_of(a.rows, kRows, 1 << 21)), block(kBlock<TPR>);
  const int64_t each = 2 * sizeof(typename IO::elem) + (a.residual ? 4 : 0) + (a.sum ? 4 : 0);
  auto go = [&](auto past) {
    hipLaunchKernelGGL((norm_fwd_kernel<IO, V, TPR, K, past>), grid, block, 0, stream, a);
  };
  with_past<V>(go, passes_cache(a.rows * a.dim * each));
}

template <class IO, class S, int V, int TPR, int K>
void bwd(const NormArgs& a, float* part, int64_t* lines, hipStream_t stream) {
  *lines = strands_of(a.rows, kBlock<TPR> / TPR);
  const dim3 grid(static_cast<unsigned>(*lines)), block(kBlock<TPR>);
  const int64_t es = sizeof(typename IO::elem);
  const int64_t each = es + sizeof(typename S::elem) + (a.dsum ? 4 : 0) + (a.dx ? es : 0) +
                       (a.dresidual ? 4 : 0);
  auto go = [&](auto past) {
    hipLaunchKernelGGL((norm_bwd_kernel<IO, S, V, TPR, K, past>), grid, block, 0, stream, a, part);
  };
  with_past<V>(go, passes_cache(a.rows * a.dim * each));
}

// Calls f with the instance's V, TPR and K: groups of four columns (V = 4) in up to four rounds (up
// to ROUNDS by 1024 threads), single columns (V = 1) in up to sixteen.  More than 64 threads take a
// row only when it has more columns than a quarter as many hold, so the fewest rounds are for 64
// alone.
template <int V, int TPR, int ROUNDS, class F>
void with_rounds(int64_t dim, F f) {
  const int64_t k = (dim + TPR * V - 1) / (TPR * V);
  using std::integral_constant;
  auto go = [&](auto kk) { f(integral_constant<int, V>{}, integral_constant<int, TPR>{}, kk); };
  if constexpr (V == 4) {
    if constexpr (TPR == 64) {
      if (k <= 1) return go(integral_constant<int, 1>{});
    }
    if (k <= 2) go(integral_constant<int, 2>{});
    else if constexpr (TPR == 1024 && ROUNDS == 3) go(integral_constant<int, 3>{});
    else if (k <= 3) go(integral_constant<int, 3>{});
    else go(integral_constant<int, 4>{});
  } else {
    if constexpr (TPR == 64) {
      if (k <= 2) return go(integral_constant<int, 2>{});
    }
    if (k <= 5) go(integral_constant<int, 5>{});
    else if constexpr (TPR == 1024) go(integral_constant<int, 8>{});
    else if (k <= 8) go(integral_constant<int, 8>{});
    else if (k <= 12) go(integral_constant<int, 12>{});
    else go(integral_constant<int, 16>{});
  }
}
template <int V, int ROUNDS, class F>
void with_threads(int64_t dim, int tpr, F f) {
  if (tpr == 64) with_rounds<V, 64, ROUNDS>(dim, f);
  else if (tpr == 256) with_rounds<V, 256, ROUNDS>(dim, f);
  else with_rounds<V, 1024, ROUNDS>(dim, f);
}
template <int ROUNDS, class F>
void with_shape(int64_t dim, bool quads, int tpr, F f) {
  if (quads) with_threads<4, ROUNDS>(dim, tpr, f);
  else with_threads<1, ROUNDS>(dim, tpr, f);
}

template <class IO>
hipError_t launch_fwd(const NormArgs& a, hipStream_t stream) {
  const uintptr_t wide = reinterpret_cast<uintptr_t>(a.residual) |
                         reinterpret_cast<uintptr_t>(a.sum) |
                         reinterpret_cast<uintptr_t>(a.weight) |
                         reinterpret_cast<uintptr_t>(a.bias);
  const uintptr_t io = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out);
  const bool quads = a.dim % 4 == 0 && wide % 16 == 0 && io % (4 * sizeof(typename IO::elem)) == 0;
  const int tpr = threads_per_row(a.dim, quads, kRoundsFwd);
  if (!tpr)
    hipLaunchKernelGGL((norm_fwd_wide_kernel<IO>), dim3(blocks_of(a.rows, 1, 4096)),
                       dim3(kWide), 0, stream, a);
  else
    with_shape<kRoundsFwd>(a.dim, quads, tpr,
                           [&](auto v, auto t, auto k) { fwd<IO, v, t, k>(a, stream); });
  return hipGetLastError();
}

template <class IO, class S>
hipError_t launch_bwd(const NormArgs& a, hipStream_t stream) {
  const uintptr_t wide = reinterpret_cast<uintptr_t>(a.dsum) |
                         reinterpret_cast<uintptr_t>(a.dresidual) |
                         reinterpret_cast<uintptr_t>(a.weight);
  const uintptr_t io = reinterpret_cast<uintptr_t>(a.dout) | reinterpret_cast<uintptr_t>(a.dx);
  const bool quads = a.dim % 4 == 0 && wide % 16 == 0 &&
                     io % (4 * sizeof(typename IO::elem)) == 0 &&
                     reinterpret_cast<uintptr_t>(a.x) % (4 * sizeof(typename S::elem)) == 0;
  const int tpr = threads_per_row(a.dim, quads, kRoundsBwd);
  float* part = a.dweight || a.dbias ? static_cast<float*>(a.workspace) : nullptr;
  int64_t lines = 0;
  if (!tpr) {
    hipLaunchKernelGGL((norm_bwd_wide_kernel<IO, S>), dim3(blocks_of(a.rows, 1, 4096)),
                       dim3(kWide), 0, stream, a);
    if (part) {
      const int64_t cols = (a.dim + 255) / 256;
      lines = a.rows < 64 ? a.rows : 64;
      hipLaunchKernelGGL((norm_param_wide_kernel<IO, S>),
                         dim3(static_cast<unsigned>(cols), static_cast<unsigned>(lines)),
                         dim3(256), 0, stream, a, part);
    }
  } else {
    with_shape<kRoundsBwd>(a.dim, quads, tpr, [&](auto v, auto t, auto k) {
      bwd<IO, S, v, t, k>(a, part, &lines, stream);
    });
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part) return e;
  ColumnSums c{};
  c.lines = lines;
  c.stride = 2 * a.dim;
  c.cols = a.dim;
  c.add(part, a.dweight, 1);
  c.add(part + a.dim, a.dbias, 1);
  return launch_column_sums(c, stream);
}

}  // namespace

size_t norm_bwd_ws_bytes(int64_t rows, int64_t dim) {
  return static_cast<size_t>((rows < kStrands ? rows : kStrands) * 2 * dim) * sizeof(float);
}

hipError_t launch_norm_fwd(const NormArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_fwd<BF16>(a, stream) : launch_fwd<F32>(a, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, bool bf16, hipStream_t stream) {
  if (!bf16) return launch_bwd<F32, F32>(a, stream);
  return a.s_f32 ? launch_bwd<BF16, F32>(a, stream) : launch_bwd<BF16, BF16>(a, stream);
}

}  // namespace ss
