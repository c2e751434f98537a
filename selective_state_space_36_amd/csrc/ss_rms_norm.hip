// ss_rms_norm.hip -- the RMS norm with a block's output scaled, dropped out and added to the
// residual stream, and the gated RMS norm in groups, with their gradients.
//
// A unit (a row, or one group of a row's columns) lies in the registers of 8 to 1024 lanes, K octs
// of columns each, so every array is read once: units of up to 16384 columns in the forward, of up
// to 8192 in the backward.  Wider ones are read again for each pass by the wide kernels, whose
// backward also reads and writes its line of sums for every unit.  Parameter gradients are otherwise
// added in registers while a workgroup walks its units, written as one line per workgroup (or unit
// place) and summed by column_sums_kernel in a fixed order.
//
// What bounds it: memory.  16384 x 2560 bf16 with residual, scale and dropout: forward 504 MB in
// 106 us (4.8 TB/s; a copy of 1 GiB reaches 5.2), backward 756 MB in 140 us (5.4, some of it from the
// 256 MB cache) and 5 us for the sums; the generator's 14 slots an element hide behind the loads.
// Gated, 16384 x 5120 bf16, z part of longer rows: backward 840 MB in 138 us behind its forward (some
// of it from the cache; 175 alone), forward 504 MB in 138 (128 alone), 3.6 TB/s and so not memory's
// rate: a workgroup loads its one row, meets at a barrier, stores and ends, with nothing on its way
// meanwhile.  One row: 2.8 us, a launch.  Non-temporal loads are kept to the backward: in the forward
// they gain 11 us and cost the backward, which finds less in the cache, 20.
//
// RMS backward alone with everything asked for, 16384 rows bf16, TB/s: 512 columns 4.6, 768 3.1, 1024
// 4.6, 2560 5.3, 4096 5.4; 5120 4.3 and 8192 4.7 with 1024 lanes' spills; 8192 rows of 12288 or 16384
// 3.2 and 3.1 (wide).  The forward is at 4.8 to 5.7 throughout.
#include "ss_head.h"
#include "ss_octs.h"
#include "ss_philox.h"
#include "ss_rows.h"

namespace ss {
namespace {

__device__ __forceinline__ float inv_root(float sumsq, float n, float eps) {
  return 1.0f / __builtin_sqrtf(sumsq / n + eps);
}

// Position of a thread: its unit place in the workgroup and its lane in the unit.
struct Place {
  int seg, lane;
};
__device__ __forceinline__ Place place(const UnitLayout& l) {
  const int seg = l.lanes > 64 ? 0 : static_cast<int>(threadIdx.x) / l.lanes;
  return Place{seg, static_cast<int>(threadIdx.x) - seg * l.lanes};
}
// The unit a place begins with, as (row, group), and its way to the next one.
struct Walk {
  int64_t u, row;
  int g;
  __device__ __forceinline__ Walk(const UnitLayout& l, int seg) {
    u = static_cast<int64_t>(blockIdx.x) * l.segs + seg;
    row = l.groups > 1 ? u / l.groups : u;
    g = static_cast<int>(u - row * l.groups);
  }
  __device__ __forceinline__ void next(const UnitLayout& l) {
    u += l.stride;
    row += l.drow;
    g += l.dg;
    if (g >= l.groups) {
      g -= l.groups;
      ++row;
    }
  }
};

// ------------------------------------------------------------------ the norm before a block

template <class IO, int K, bool DROP>
__global__ __launch_bounds__(1024) void rms_fwd_kernel(RmsArgs p, UnitLayout l) {
  using E = typename IO::elem;
  __shared__ float lds[2 * 16];
  const Place at = place(l);
  const float n = static_cast<float>(l.width);
  PhiloxKey key{};
  if constexpr (DROP) key = philox_key(p.drop.rng);
  int phase = 0;
  for (Walk w(l, at.seg); w.u < l.units; w.next(l)) {
    const int64_t base = w.row * l.width;
    float v[K][8], r[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * l.lanes + at.lane) * 8, left = l.width - c;
      load8<IO>(static_cast<const E*>(p.x) + base + c, left, v[k]);
      if (p.residual) load8<F32>(p.residual + base + c, left, r[k]);
    }
    if (p.branch) {
      float sq[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) sq[0] = fmaf(v[k][j], v[k][j], sq[0]);
      unit_sums<1>(sq, l.lanes, lds, phase++);
      const float rb = inv_root(sq[0], n, p.eps);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] *= rb;
      if (at.lane == 0 && p.branch_rstd) p.branch_rstd[w.row] = rb;
    }
    float sq[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * l.lanes + at.lane) * 8, left = l.width - c;
      if (p.scale) {
        float s[8];
        load8<F32>(p.scale + c, left, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] *= s[j];
      }
      if constexpr (DROP)
        drop8(v[k], keep8(key, c >> 3, static_cast<uint32_t>(w.row), p.drop.cut), p.drop.up);
      if (p.residual) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] += r[k][j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sq[0] = fmaf(v[k][j], v[k][j], sq[0]);
      if (p.sum) store8<F32>(p.sum + base + c, left, v[k]);
    }
    unit_sums<1>(sq, l.lanes, lds, phase++);
    const float rstd = inv_root(sq[0], n, p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * l.lanes + at.lane) * 8, left = l.width - c;
      float o[8];
      if (p.weight) {
        load8<F32>(p.weight + c, left, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= v[k][j] * rstd;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = v[k][j] * rstd;
      }
      store8<IO>(static_cast<E*>(p.out) + base + c, left, o);
    }
    if (at.lane == 0 && p.rstd) p.rstd[w.row] = rstd;
  }
}

// Where a place's parameter sums go: its line of `part` (cols columns a line), group g's columns.
// One line per place that shares the group with no other of its workgroup; with a single group the
// places of a workgroup are first added in order through LDS, and it writes one line.
template <int N>
__device__ __forceinline__ void write_lines(float (&acc)[N][8], const UnitLayout& l,
                                            const Place& at, int g, int64_t cols, float* part,
                                            float* fold) {
  int64_t line;
  if (l.groups == 1) {
    line = blockIdx.x;
    if (l.segs > 1) {
      const int per = l.lanes * 8;  // floats a place holds of one sum
#pragma unroll
      for (int q = 0; q < N; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          fold[(at.seg * N + q) * per + j * l.lanes + at.lane] = acc[q][j];
      __syncthreads();
      if (at.seg) return;
      for (int s = 1; s < l.segs; ++s)
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc[q][j] += fold[(s * N + q) * per + j * l.lanes + at.lane];
    }
  } else {
    line = (static_cast<int64_t>(blockIdx.x) * l.segs + at.seg) / l.groups;
  }
  const int c = at.lane * 8;
#pragma unroll
  for (int q = 0; q < N; ++q)
    store8<F32>(part + (line * N + q) * cols + static_cast<int64_t>(g) * l.width + c, l.width - c,
                acc[q]);
}

// One oct per lane: a place's sums, its row and the next one take about 140 registers.  (The next
// row asked for ahead: 210 -> 140 us at 16384 x 2560 bf16, where its rows are not spilled: MOST 512,
// for up to 4096 columns; with 1024 lanes the compiler has 128 registers and spills 1 to 24, 16 for
// bf16 with a float32 sum and dropout.)  Rows of over 8192 columns go to the wide kernels.
template <class IO, class S, bool DROP, bool PAST, int MOST>
__global__ __launch_bounds__(MOST) void rms_bwd_kernel(RmsArgs p, UnitLayout l, float* part) {
  using E = typename IO::elem;
  __shared__ float lds[2 * 16];
  __shared__ float fold[256 * 2 * 8];
  const Place at = place(l);
  const float inv = 1.0f / static_cast<float>(l.width);
  const int c = at.lane * 8, left = l.width - c;
  PhiloxKey key{};
  if constexpr (DROP) key = philox_key(p.drop.rng);
  float acc[2][8] = {};  // dweight, dscale
  float wt[8], sc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) wt[j] = sc[j] = 1.0f;
  if (p.weight) load8<F32>(p.weight + c, left, wt);
  if (p.scale) load8<F32>(p.scale + c, left, sc);
  // The next row is asked for before this one's sums.
  Oct<IO> go, xo;
  Oct<S> so;
  Oct<F32> uo;
  float rstd = 0.0f, rb = 1.0f;
  auto fetch = [&](int64_t row, int n) {
    const int64_t base = row * l.width;
    go = load_oct<IO, PAST>(static_cast<const E*>(p.dout) + base + c, n);
    so = load_oct<S, PAST>(static_cast<const typename S::elem*>(p.s) + base + c, n);
    if (p.x) xo = load_oct<IO, PAST>(static_cast<const E*>(p.x) + base + c, n);
    if (p.dsum) uo = load_oct<F32, PAST>(p.dsum + base + c, n);
    rstd = p.rstd_in[row];
    if (p.branch) rb = p.branch_rstd_in[row];
  };
  int phase = 0;
  Walk w(l, at.seg);
  if (w.u < l.units) fetch(w.row, left);
  while (w.u < l.units) {
    const int64_t row = w.row, base = row * l.width;
    float sh[8], g[8], x[8], u[8], c1[1] = {0.0f};
    const float rs = rstd, rbs = rb;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = go[j];
      sh[j] = so[j] * rs;
      x[j] = p.x ? xo[j] * rbs : 0.0f;
      u[j] = p.dsum ? uo[j] : 0.0f;
    }
    w.next(l);
    if (w.u < l.units) fetch(w.row, left);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[0][j] = fmaf(g[j], sh[j], acc[0][j]);
      g[j] *= wt[j];
      c1[0] = fmaf(g[j], sh[j], c1[0]);
    }
    unit_sums<1>(c1, l.lanes, lds, phase++);
    const float m1 = c1[0] * inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = fmaf(rs, fmaf(-sh[j], m1, g[j]), u[j]);
    if (p.dresidual) store8<F32>(p.dresidual + base + c, left, g);
    uint32_t keep = 0xff;
    if constexpr (DROP) {
      keep = keep8(key, at.lane, static_cast<uint32_t>(row), p.drop.cut);
      drop8(g, keep, p.drop.up);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // (a dropped x is no factor, whatever it is)
      if (!DROP || keep >> j & 1) acc[1][j] = fmaf(g[j], x[j], acc[1][j]);
      g[j] *= sc[j];
    }
    if (p.branch) {
      float c2[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < 8; ++j) c2[0] = fmaf(g[j], x[j], c2[0]);
      unit_sums<1>(c2, l.lanes, lds, phase++);
      const float m2 = c2[0] * inv;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = rbs * fmaf(-x[j], m2, g[j]);
    }
    if (p.dx) store8<IO>(static_cast<E*>(p.dx) + base + c, left, g);
  }
  if (part) write_lines<2>(acc, l, at, 0, l.width, part, fold);
}

// ------------------------------------------------------------------ the gated norm

template <class IO, int K, bool FIRST>
__global__ __launch_bounds__(1024) void gated_norm_fwd_kernel(GatedNormArgs p, UnitLayout l) {
  using E = typename IO::elem;
  __shared__ float lds[2 * 16];
  const Place at = place(l);
  const float n = static_cast<float>(l.width);
  int phase = 0;
  for (Walk w(l, at.seg); w.u < l.units; w.next(l)) {
    const int64_t col = static_cast<int64_t>(w.g) * l.width;
    const int64_t base = w.row * p.dim + col, zbase = w.row * p.z_stride + col;
    float v[K][8], z[K][8], sq[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * l.lanes + at.lane) * 8, left = l.width - c;
      load8<IO>(static_cast<const E*>(p.x) + base + c, left, v[k]);
      if (p.z) load8<IO>(static_cast<const E*>(p.z) + zbase + c, left, z[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (p.z) z[k][j] *= sigmoid_f(z[k][j]);
        if (FIRST && p.z) v[k][j] *= z[k][j];
        sq[0] = fmaf(v[k][j], v[k][j], sq[0]);
      }
    unit_sums<1>(sq, l.lanes, lds, phase++);
    const float rstd = inv_root(sq[0], n, p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * l.lanes + at.lane) * 8, left = l.width - c;
      float wt[8];
      if (p.weight) load8<F32>(p.weight + col + c, left, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[k][j] *= rstd;
        if (p.weight) v[k][j] *= wt[j];
        if (!FIRST && p.z) v[k][j] *= z[k][j];
      }
      store8<IO>(static_cast<E*>(p.out) + base + c, left, v[k]);
    }
    if (at.lane == 0 && p.rstd) p.rstd[w.u] = rstd;
  }
}

template <class IO, bool FIRST, bool PAST>
__global__ __launch_bounds__(1024) void gated_norm_bwd_kernel(GatedNormArgs p, UnitLayout l,
                                                              float* part) {
  using E = typename IO::elem;
  __shared__ float lds[2 * 16];
  __shared__ float fold[256 * 8];
  const Place at = place(l);
  const float inv = 1.0f / static_cast<float>(l.width);
  const int c = at.lane * 8, left = l.width - c;
  float acc[1][8] = {};
  int phase = 0;
  Walk w(l, at.seg);
  const int g0 = w.g;  // a place keeps its group (launch: stride is a multiple of the groups)
  const int64_t col = static_cast<int64_t>(g0) * l.width + c;
  float wt[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) wt[j] = 1.0f;
  if (p.weight) load8<F32>(p.weight + col, left, wt);
  Oct<IO> xo, zo, go;
  float rstd = 0.0f;
  auto fetch = [&]() {
    const int64_t base = w.row * p.dim + col;
    go = load_oct<IO, PAST>(static_cast<const E*>(p.dout) + base, left);
    xo = load_oct<IO, PAST>(static_cast<const E*>(p.x) + base, left);
    if (p.z) zo = load_oct<IO, PAST>(static_cast<const E*>(p.z) + w.row * p.z_stride + col, left);
    rstd = p.rstd_in[w.u];
  };
  if (w.u < l.units) fetch();
  while (w.u < l.units) {
    const int64_t base = w.row * p.dim + col;
    // FIRST: u = x silu(z), hat = u rstd, out = hat w.   Else: hat = x rstd, out = hat w silu(z).
    // hat and g = w d (silu(z)) stay; of dx = du gate and dz the factors x (or d hat w), gate, slope
    float hat[8], g[8], gate[8], side[8], c1[1] = {0.0f};
    const float rs = rstd;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = go[j], x = xo[j], zz = p.z ? zo[j] : 0.0f;
      const float sg = p.z ? sigmoid_f(zz) : 1.0f;
      const float slope = sg * fmaf(zz, 1.0f - sg, 1.0f);
      gate[j] = p.z ? zz * sg : 1.0f;
      hat[j] = x * rs * (FIRST ? gate[j] : 1.0f);
      const float after = FIRST ? d : d * gate[j];
      side[j] = (FIRST ? x : d * hat[j] * wt[j]) * slope;
      acc[0][j] = fmaf(after, hat[j], acc[0][j]);
      g[j] = after * wt[j];
      c1[0] = fmaf(g[j], hat[j], c1[0]);
    }
    w.next(l);
    if (w.u < l.units) fetch();
    unit_sums<1>(c1, l.lanes, lds, phase++);
    const float m1 = c1[0] * inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float du = rs * fmaf(-hat[j], m1, g[j]);
      g[j] = FIRST ? du * gate[j] : du;
      if (FIRST) side[j] *= du;
    }
    store8<IO>(static_cast<E*>(p.dx) + base, left, g);
    if (p.z) store8<IO>(static_cast<E*>(p.dz) + base, left, side);
  }
  if (part) write_lines<1>(acc, l, at, g0, p.dim, part, fold);
}

// ------------------------------------------------------------------ units too wide for registers

constexpr int kWide = 1024;

// Calls f(column, columns left) for this thread's octs of a unit.
template <class F>
__device__ __forceinline__ void each_oct(int width, F f) {
  for (int64_t c = threadIdx.x * 8ll; c < width; c += kWide * 8ll)
    f(static_cast<int>(c), static_cast<int>(width - c));
}

template <class IO, bool DROP>
__global__ __launch_bounds__(kWide) void rms_fwd_wide_kernel(RmsArgs p, UnitLayout l) {
  using E = typename IO::elem;
  __shared__ float lds[2 * 16];
  const float n = static_cast<float>(l.width);
  PhiloxKey key{};
  if constexpr (DROP) key = philox_key(p.drop.rng);
  int phase = 0;
  for (int64_t row = blockIdx.x; row < l.units; row += gridDim.x) {
    const int64_t base = row * l.width;
    float rb = 1.0f;
    if (p.branch) {
      float sq[1] = {0.0f};
      each_oct(l.width, [&](int c, int left) {
        float v[8];
        load8<IO>(static_cast<const E*>(p.x) + base + c, left, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sq[0] = fmaf(v[j], v[j], sq[0]);
      });
      unit_sums<1>(sq, kWide, lds, phase++);
      rb = inv_root(sq[0], n, p.eps);
      if (threadIdx.x == 0 && p.branch_rstd) p.branch_rstd[row] = rb;
    }
    auto value = [&](int c, int left, float (&v)[8]) {
      load8<IO>(static_cast<const E*>(p.x) + base + c, left, v);
      float s[8];
      if (p.scale) load8<F32>(p.scale + c, left, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= p.scale ? rb * s[j] : rb;
      if constexpr (DROP)
        drop8(v, keep8(key, c >> 3, static_cast<uint32_t>(row), p.drop.cut), p.drop.up);
      if (p.residual) {
        load8<F32>(p.residual + base + c, left, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += s[j];
      }
    };
    float sq[1] = {0.0f};
    each_oct(l.width, [&](int c, int left) {
      float v[8];
      value(c, left, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sq[0] = fmaf(v[j], v[j], sq[0]);
    });
    unit_sums<1>(sq, kWide, lds, phase++);
    const float rstd = inv_root(sq[0], n, p.eps);
    each_oct(l.width, [&](int c, int left) {
      float v[8], o[8];
      value(c, left, v);
      if (p.sum) store8<F32>(p.sum + base + c, left, v);
      if (p.weight) load8<F32>(p.weight + c, left, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = p.weight ? o[j] * (v[j] * rstd) : v[j] * rstd;
      store8<IO>(static_cast<E*>(p.out) + base + c, left, o);
    });
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
  }
}

// Adds v to this workgroup's line (its first unit writes it).
__device__ __forceinline__ void add_line(float* line, int left, float (&v)[8], bool first) {
  if (!first) {
    float o[8];
    load8<F32>(line, left, o);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += o[j];
  }
  store8<F32>(line, left, v);
}

template <class IO, class S, bool DROP>
__global__ __launch_bounds__(kWide) void rms_bwd_wide_kernel(RmsArgs p, UnitLayout l,
                                                             float* part) {
  using E = typename IO::elem;
  __shared__ float lds[2 * 16];
  const float inv = 1.0f / static_cast<float>(l.width);
  PhiloxKey key{};
  if constexpr (DROP) key = philox_key(p.drop.rng);
  int phase = 0;
  for (int64_t row = blockIdx.x; row < l.units; row += gridDim.x) {
    const int64_t base = row * l.width;
    const bool first = row == blockIdx.x;
    const float rstd = p.rstd_in[row];
    const float rb = p.branch ? p.branch_rstd_in[row] : 1.0f;
    float* line = part ? part + static_cast<int64_t>(blockIdx.x) * 2 * l.width : nullptr;
    auto load = [&](int c, int left, float (&g)[8], float (&sh)[8]) {
      load8<IO>(static_cast<const E*>(p.dout) + base + c, left, g);
      load8<S>(static_cast<const typename S::elem*>(p.s) + base + c, left, sh);
#pragma unroll
      for (int j = 0; j < 8; ++j) sh[j] *= rstd;
    };
    auto weigh = [&](const float* by, int c, int left, float (&g)[8]) {
      if (!by) return;
      float w[8];
      load8<F32>(by + c, left, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] *= w[j];
    };
    float c1[1] = {0.0f};
    each_oct(l.width, [&](int c, int left) {
      float g[8], sh[8], dw[8];
      load(c, left, g, sh);
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[j] = g[j] * sh[j];
      if (line) add_line(line + c, left, dw, first);
      weigh(p.weight, c, left, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) c1[0] = fmaf(g[j], sh[j], c1[0]);
    });
    unit_sums<1>(c1, kWide, lds, phase++);
    const float m1 = c1[0] * inv;
    // the sum's gradient, then (dropped) the branch's
    auto dsum = [&](int c, int left, float (&g)[8]) {
      float sh[8], u[8];
      load(c, left, g, sh);
      weigh(p.weight, c, left, g);
      if (p.dsum) load8<F32>(p.dsum + base + c, left, u);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        g[j] = fmaf(rstd, fmaf(-sh[j], m1, g[j]), p.dsum ? u[j] : 0.0f);
    };
    auto drop = [&](int c, float (&g)[8]) {
      uint32_t keep = 0xff;
      if constexpr (DROP) {
        keep = keep8(key, c >> 3, static_cast<uint32_t>(row), p.drop.cut);
        drop8(g, keep, p.drop.up);
      }
      return keep;
    };
    auto hat = [&](int c, int left, float (&x)[8]) {
      load8<IO>(static_cast<const E*>(p.x) + base + c, left, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= rb;
    };
    float m2 = 0.0f;
    if (p.branch) {
      float c2[1] = {0.0f};
      each_oct(l.width, [&](int c, int left) {
        float g[8], x[8];
        dsum(c, left, g);
        drop(c, g);
        weigh(p.scale, c, left, g);
        hat(c, left, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) c2[0] = fmaf(g[j], x[j], c2[0]);
      });
      unit_sums<1>(c2, kWide, lds, phase++);
      m2 = c2[0] * inv;
    }
    each_oct(l.width, [&](int c, int left) {
      float g[8], x[8], ds[8];
      dsum(c, left, g);
      if (p.dresidual) store8<F32>(p.dresidual + base + c, left, g);
      const uint32_t keep = drop(c, g);
      if (p.x) {
        hat(c, left, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) ds[j] = keep >> j & 1 ? g[j] * x[j] : 0.0f;
        if (line) add_line(line + l.width + c, left, ds, first);
      }
      weigh(p.scale, c, left, g);
      if (p.branch) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = rb * fmaf(-x[j], m2, g[j]);
      }
      if (p.dx) store8<IO>(static_cast<E*>(p.dx) + base + c, left, g);
    });
  }
}

// One workgroup per unit, each of its group alone (the launch's grid is a multiple of the groups).
template <class IO, bool FIRST>
__global__ __launch_bounds__(kWide) void gated_norm_fwd_wide_kernel(GatedNormArgs p,
                                                                    UnitLayout l) {
  using E = typename IO::elem;
  __shared__ float lds[2 * 16];
  const float n = static_cast<float>(l.width);
  int phase = 0;
  for (Walk w(l, 0); w.u < l.units; w.next(l)) {
    const int64_t col = static_cast<int64_t>(w.g) * l.width;
    const int64_t base = w.row * p.dim + col, zbase = w.row * p.z_stride + col;
    auto load = [&](int c, int left, float (&v)[8], float (&z)[8]) {
      load8<IO>(static_cast<const E*>(p.x) + base + c, left, v);
      if (!p.z) return;
      load8<IO>(static_cast<const E*>(p.z) + zbase + c, left, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[j] *= sigmoid_f(z[j]);
        if (FIRST) v[j] *= z[j];
      }
    };
    float sq[1] = {0.0f};
    each_oct(l.width, [&](int c, int left) {
      float v[8], z[8];
      load(c, left, v, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) sq[0] = fmaf(v[j], v[j], sq[0]);
    });
    unit_sums<1>(sq, kWide, lds, phase++);
    const float rstd = inv_root(sq[0], n, p.eps);
    each_oct(l.width, [&](int c, int left) {
      float v[8], z[8], wt[8];
      load(c, left, v, z);
      if (p.weight) load8<F32>(p.weight + col + c, left, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] *= rstd;
        if (p.weight) v[j] *= wt[j];
        if (!FIRST && p.z) v[j] *= z[j];
      }
      store8<IO>(static_cast<E*>(p.out) + base + c, left, v);
    });
    if (threadIdx.x == 0 && p.rstd) p.rstd[w.u] = rstd;
  }
}

template <class IO, bool FIRST>
__global__ __launch_bounds__(kWide) void gated_norm_bwd_wide_kernel(GatedNormArgs p, UnitLayout l,
                                                                    float* part) {
  using E = typename IO::elem;
  __shared__ float lds[2 * 16];
  const float inv = 1.0f / static_cast<float>(l.width);
  int phase = 0;
  Walk w(l, 0);
  const int64_t col = static_cast<int64_t>(w.g) * l.width;
  float* line = part ? part + blockIdx.x / l.groups * p.dim + col : nullptr;
  for (bool first = true; w.u < l.units; w.next(l), first = false) {
    const int64_t base = w.row * p.dim + col, zbase = w.row * p.z_stride + col;
    const float rstd = p.rstd_in[w.u];
    auto load = [&](int c, int left, float (&d)[8], float (&x)[8], float (&z)[8], float (&wt)[8]) {
      load8<IO>(static_cast<const E*>(p.dout) + base + c, left, d);
      load8<IO>(static_cast<const E*>(p.x) + base + c, left, x);
      if (p.z) load8<IO>(static_cast<const E*>(p.z) + zbase + c, left, z);
      if (p.weight) load8<F32>(p.weight + col + c, left, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!p.z) z[j] = 0.0f;
        if (!p.weight) wt[j] = 1.0f;
      }
    };
    float c1[1] = {0.0f};
    each_oct(l.width, [&](int c, int left) {
      float d[8], x[8], z[8], wt[8], dw[8];
      load(c, left, d, x, z, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gate = p.z ? z[j] * sigmoid_f(z[j]) : 1.0f;
        const float hat = x[j] * rstd * (FIRST ? gate : 1.0f);
        const float after = FIRST ? d[j] : d[j] * gate;
        dw[j] = after * hat;
        c1[0] = fmaf(after * wt[j], hat, c1[0]);
      }
      if (line) add_line(line + c, left, dw, first);
    });
    unit_sums<1>(c1, kWide, lds, phase++);
    const float m1 = c1[0] * inv;
    each_oct(l.width, [&](int c, int left) {
      float d[8], x[8], z[8], wt[8], dx[8], dz[8];
      load(c, left, d, x, z, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float sg = p.z ? sigmoid_f(z[j]) : 1.0f;
        const float gate = p.z ? z[j] * sg : 1.0f;
        const float slope = sg * fmaf(z[j], 1.0f - sg, 1.0f);
        const float hat = x[j] * rstd * (FIRST ? gate : 1.0f);
        const float after = FIRST ? d[j] : d[j] * gate;
        const float du = rstd * fmaf(-hat, m1, after * wt[j]);
        dx[j] = FIRST ? du * gate : du;
        dz[j] = (FIRST ? du * x[j] : d[j] * hat * wt[j]) * slope;
      }
      store8<IO>(static_cast<E*>(p.dx) + base + c, left, dx);
      if (p.z) store8<IO>(static_cast<E*>(p.dz) + base + c, left, dz);
    });
  }
}

// ------------------------------------------------------------------ launches

struct Shape {
  UnitLayout l;
  int k, threads, blocks;
};

constexpr int64_t kFwdBlocks = 1 << 20;
// Workgroups, and so lines of sums, of the backward.  Few rows: one each as long as the lines are
// few (1001 x 1027 f32, 1001 workgroups 12.3 + 5.2 us for the sums, 256 of four rows 18.1 + 3.9).
// Many: about as many workgroups as run at once at 2560 columns, five waves each (16384 x 2560 bf16,
// 512 workgroups 140 + 4.7 us, 1024 144 + 5.2, 3276 196 + 14).  Rows of 520 to 1024 columns are two
// waves, of which 512 leave two thirds of the places empty; the number was not tried there.
constexpr int64_t kFewRowsBlocks = 1024, kManyRowsBlocks = 512;

int64_t gcd(int64_t a, int64_t b) { return b ? gcd(b, a % b) : a; }

// Lanes, octs per lane and workgroups for `rows` rows of `groups` groups of `width` columns: an oct
// a lane, in the forward two where 1024 lanes are not enough.  Backward: a place keeps its group,
// and the workgroups are few enough for their lines of sums.
Shape shape_of(int64_t rows, int64_t groups, int64_t width, bool backward) {
  Shape s{};
  const int64_t octs = (width + 7) / 8;
  s.l.groups = static_cast<int32_t>(groups);
  s.l.width = static_cast<int32_t>(width);
  s.l.units = rows * groups;
  s.k = octs <= 1024 ? 1 : octs <= 2048 && !backward ? 2 : 0;
  if (s.k == 0) {
    s.l.lanes = s.threads = kWide;
  } else if (octs <= 64) {
    s.l.lanes = 8;
    while (s.l.lanes < octs) s.l.lanes *= 2;
    s.threads = 256;
  } else {
    s.l.lanes = s.threads = static_cast<int>(((octs + s.k - 1) / s.k + 63) / 64 * 64);
  }
  s.l.segs = s.l.lanes > 64 ? 1 : s.threads / s.l.lanes;
  int64_t blocks = (s.l.units + s.l.segs - 1) / s.l.segs;
  if (backward) {
    const int64_t cap = blocks > 4096 ? kManyRowsBlocks : kFewRowsBlocks;
    if (blocks > cap) blocks = cap;
    const int64_t step = groups / gcd(groups, s.l.segs);
    blocks = (blocks + step - 1) / step * step;
  } else if (blocks > kFwdBlocks) {
    blocks = kFwdBlocks;
  }
  s.blocks = static_cast<int>(blocks);
  s.l.stride = blocks * s.l.segs;
  s.l.drow = s.l.stride / groups;
  s.l.dg = static_cast<int32_t>(s.l.stride - s.l.drow * groups);
  return s;
}

Shape rms_bwd_shape(int64_t rows, int64_t dim) { return shape_of(rows, 1, dim, true); }
Shape gated_bwd_shape(int64_t rows, int64_t dim, int64_t groups) {
  return shape_of(rows, groups, dim / groups, true);
}
int64_t gated_lines(const Shape& s) { return s.l.groups == 1 ? s.blocks : s.l.drow; }

template <class F>
void with_io(bool bf16, F f) {
  if (bf16) f(BF16{});
  else f(F32{});
}

}  // namespace

size_t rms_bwd_ws_bytes(int64_t rows, int64_t dim) {
  return static_cast<size_t>(rms_bwd_shape(rows, dim).blocks) * 2 * dim * sizeof(float);
}

hipError_t launch_rms_fwd(const RmsArgs& a, bool bf16, hipStream_t stream) {
  const Shape s = shape_of(a.rows, 1, a.dim, false);
  with_io(bf16, [&](auto io) {
    using IO = decltype(io);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(s.blocks), dim3(s.threads), 0, stream, a, s.l);
    };
    if (a.drop.rng) {
      if (s.k == 0) go(rms_fwd_wide_kernel<IO, true>);
      else if (s.k == 1) go(rms_fwd_kernel<IO, 1, true>);
      else go(rms_fwd_kernel<IO, 2, true>);
    } else {
      if (s.k == 0) go(rms_fwd_wide_kernel<IO, false>);
      else if (s.k == 1) go(rms_fwd_kernel<IO, 1, false>);
      else go(rms_fwd_kernel<IO, 2, false>);
    }
  });
  return hipGetLastError();
}

hipError_t launch_rms_bwd(const RmsArgs& a, bool bf16, hipStream_t stream) {
  const Shape s = rms_bwd_shape(a.rows, a.dim);
  float* part = a.dweight || a.dscale ? a.workspace : nullptr;
  const int64_t es = bf16 ? 2 : 4, n = a.rows * a.dim;
  const bool past =
      passes_cache(n * (es + (a.s_f32 ? 4 : es) + (a.x ? es : 0) + (a.dsum ? 4 : 0) +
                        (a.dx ? es : 0) + (a.dresidual ? 4 : 0)));
  auto run = [&](auto io, auto sv) {
    using IO = decltype(io);
    using S = decltype(sv);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(s.blocks), dim3(s.threads), 0, stream, a, s.l, part);
    };
    with_bools([&](auto drop, auto nt) {
      constexpr bool D = decltype(drop)::value, T = decltype(nt)::value;
      if (s.k == 0) go(rms_bwd_wide_kernel<IO, S, D>);
      else if (s.threads <= 512) go(rms_bwd_kernel<IO, S, D, T, 512>);
      else go(rms_bwd_kernel<IO, S, D, T, 1024>);
    }, a.drop.rng != nullptr, past);
  };
  if (!bf16) run(F32{}, F32{});
  else if (a.s_f32) run(BF16{}, F32{});
  else run(BF16{}, BF16{});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part) return e;
  ColumnSums c{};
  c.lines = s.blocks;
  c.stride = 2 * a.dim;
  c.cols = a.dim;
  c.add(part, a.dweight, 1);
  c.add(part + a.dim, a.dscale, 1);
  return launch_column_sums(c, stream);
}

size_t gated_norm_bwd_ws_bytes(int64_t rows, int64_t dim, int64_t groups) {
  return static_cast<size_t>(gated_lines(gated_bwd_shape(rows, dim, groups))) * dim *
         sizeof(float);
}

hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, bool bf16, hipStream_t stream) {
  const Shape s = shape_of(a.rows, a.groups, a.dim / a.groups, false);
  with_io(bf16, [&](auto io) {
    using IO = decltype(io);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(s.blocks), dim3(s.threads), 0, stream, a, s.l);
    };
    if (a.gate_first) {
      if (s.k == 0) go(gated_norm_fwd_wide_kernel<IO, true>);
      else if (s.k == 1) go(gated_norm_fwd_kernel<IO, 1, true>);
      else go(gated_norm_fwd_kernel<IO, 2, true>);
    } else {
      if (s.k == 0) go(gated_norm_fwd_wide_kernel<IO, false>);
      else if (s.k == 1) go(gated_norm_fwd_kernel<IO, 1, false>);
      else go(gated_norm_fwd_kernel<IO, 2, false>);
    }
  });
  return hipGetLastError();
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, bool bf16, hipStream_t stream) {
  const Shape s = gated_bwd_shape(a.rows, a.dim, a.groups);
  float* part = a.dweight ? a.workspace : nullptr;
  const bool past = passes_cache(a.rows * a.dim * (bf16 ? 2 : 4) * (a.z ? 5 : 3));
  with_io(bf16, [&](auto io) {
    using IO = decltype(io);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(s.blocks), dim3(s.threads), 0, stream, a, s.l, part);
    };
    with_bools([&](auto first, auto nt) {
      constexpr bool G = decltype(first)::value, T = decltype(nt)::value;
      if (s.k == 0) go(gated_norm_bwd_wide_kernel<IO, G>);
      else go(gated_norm_bwd_kernel<IO, G, T>);
    }, a.gate_first, past);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part) return e;
  ColumnSums c{};
  c.lines = gated_lines(s);
  c.stride = c.cols = a.dim;
  c.add(part, a.dweight, 1);
  return launch_column_sums(c, stream);
}

}  // namespace ss
