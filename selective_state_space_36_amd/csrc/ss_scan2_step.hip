// ss_scan2_step.hip -- one token of the multi-head scan, and of the convolution in front of it.
//
//     S[n,p] <- exp(dt A) S[n,p] + dt B[n] x[p];   out[p] = (sum_n C[n] S[n,p] + D x[p]) silu(z[p])
//
// One workgroup per (batch row, head, block of channels): TP lanes of V channels side by side,
// 256 / TP rows of states, every state read and written once.  The sums over the states run over
// the lanes of a wave by shuffles, over the waves through LDS.
//
// The convolution's window of B and C is shared by all heads of a group, and it is shifted in
// place, so it is a kernel of its own in front of this one: x, B and C cross in float32 (the
// workspace), unrounded.
//
// What bounds it: memory.  128 rows of 80 heads x 128 x 64: 671 MB of states in 115 us (5.8 TB/s,
// non-temporal; four channels a lane, eight states of a lane in flight), the convolution's kernel 9
// (two channels a lane the same: it waits for a window that nothing has left in a cache).  One row:
// 5.9 us and 3.4 (latency; in 16-channel blocks, 320 workgroups), below the 15 us of the call on the
// host.
#include "ss_head.h"
#include "ss_octs.h"
#include "ss_rows.h"

namespace ss {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kAhead = 8;  // states of a lane in flight

template <class IO>
__global__ __launch_bounds__(kThreads) void conv_act_kernel(Scan2StepArgs p) {
  using E = typename IO::elem;
  const int64_t d = p.conv_dim;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.batch * d) return;
  const int64_t b = i / d, c = i - b * d;
  const int k = p.conv_k;
  E* st = static_cast<E*>(p.conv_state) + b * (k - 1) * d + c;
  const E now = static_cast<const E*>(p.xbc)[b * p.xbc_stride + c];
  const float* w = p.conv_weight + c * k;
  float v = p.conv_bias ? p.conv_bias[c] : 0.0f;
  E prev[3];
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < k - 1) prev[j] = st[j * d];
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < k - 1) v = fmaf(w[j], IO::widen(prev[j]), v);
  v = fmaf(w[k - 1], IO::widen(now), v);
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (j < k - 2) st[j * d] = prev[j + 1];
  if (k > 1) st[(k - 2) * d] = now;
  p.act[i] = silu_f(v);
}

// IO: dt, z and out; XT: x, B and C (float32 behind the convolution).
template <class IO, class XT, int V, int TP, bool PAST>
__global__ __launch_bounds__(kThreads) void scan2_step_kernel(Scan2StepArgs p) {
  using E = typename IO::elem;
  using X = typename XT::elem;
  typedef float vec __attribute__((ext_vector_type(V)));
  constexpr int kRows = kThreads / TP;
  __shared__ float part[kWaves][TP * V];
  const int P = p.headdim, N = p.d_state;
  int64_t w = blockIdx.x;
  const int pb = static_cast<int>(w % p.n_pblk);
  w /= p.n_pblk;
  const int64_t b = w / p.nheads, h = w - b * p.nheads, grp = h / (p.nheads / p.ngroups);
  const int tp = threadIdx.x % TP, row = threadIdx.x / TP;
  const int c0 = (pb * TP + tp) * V;  // V divides P, so a lane has all of its channels or none
  const bool live = c0 < P;
  float* S = p.state + (b * p.nheads + h) * N * P + c0;
  const X* Bp = static_cast<const X*>(p.B) + b * p.b_stride + grp * N;
  const X* Cp = static_cast<const X*>(p.C) + b * p.c_stride + grp * N;
  const X* xp = static_cast<const X*>(p.x) + b * p.x_stride + h * P + c0;

  const float raw = IO::widen(static_cast<const E*>(p.dt)[b * p.dt_stride + h]) +
                    (p.dt_bias ? p.dt_bias[h] : 0.0f);
  float x[V], y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    x[v] = live ? XT::widen(xp[v]) : 0.0f;
    y[v] = 0.0f;
  }
  const float dt = p.softplus ? softplus_f(raw) : raw;
  const float decay = exp2_hw(dt * (p.A[h] * kLog2e));
  for (int n0 = row; n0 < N; n0 += kRows * kAhead) {
    vec s[kAhead];
    float bn[kAhead], cn[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int n = n0 + k * kRows;
      if (n < N) {
        if (live) {
          const vec* at = reinterpret_cast<const vec*>(S + static_cast<int64_t>(n) * P);
          s[k] = PAST ? __builtin_nontemporal_load(at) : *at;
        }
        bn[k] = XT::widen(Bp[n]);
        cn[k] = XT::widen(Cp[n]);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int n = n0 + k * kRows;
      if (n < N && live) {
        const float in = dt * bn[k];
        vec t;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          t[v] = fmaf(in, x[v], decay * s[k][v]);
          y[v] = fmaf(cn[k], t[v], y[v]);
        }
        vec* at = reinterpret_cast<vec*>(S + static_cast<int64_t>(n) * P);
        if constexpr (PAST) __builtin_nontemporal_store(t, at);
        else *at = t;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int off = TP; off < 64; off *= 2) y[v] += __shfl_xor(y[v], off);
  if ((threadIdx.x & 63) < TP) {
#pragma unroll
    for (int v = 0; v < V; ++v) part[threadIdx.x >> 6][tp * V + v] = y[v];
  }
  __syncthreads();
  const int c = threadIdx.x, col = pb * TP * V + c;
  if (c < TP * V && col < P) {
    float s = part[0][c];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) s += part[k][c];
    const float xc = XT::widen(static_cast<const X*>(p.x)[b * p.x_stride + h * P + col]);
    s = fmaf(p.D ? p.D[h] : 0.0f, xc, s);
    if (p.z)
      s *= silu_f(IO::widen(static_cast<const E*>(p.z)[b * p.z_stride + h * P + col]));
    static_cast<E*>(p.out)[(b * p.nheads + h) * P + col] = IO::from_float(s);
  }
}

template <class IO, class XT>
hipError_t launch(Scan2StepArgs a, hipStream_t stream) {
  const int64_t heads = a.batch * a.nheads;
  const int64_t state = heads * a.d_state * a.headdim * 4;
  // Four channels a lane where the rows of the state are whole 16-byte pieces.
  const bool wide = a.headdim % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
  auto go = [&](auto kernel, int cols) {
    a.n_pblk = (a.headdim + cols - 1) / cols;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(heads * a.n_pblk)), dim3(kThreads), 0,
                       stream, a);
    return hipGetLastError();
  };
  // Few heads: blocks of 16 channels, so that four times as many workgroups share the work.
  const bool few = heads < 512;
  if (wide) {
    if (few) return go(scan2_step_kernel<IO, XT, 4, 4, false>, 16);
    if (passes_cache(2 * state)) return go(scan2_step_kernel<IO, XT, 4, 16, true>, 64);
    return go(scan2_step_kernel<IO, XT, 4, 16, false>, 64);
  }
  if (few) return go(scan2_step_kernel<IO, XT, 1, 16, false>, 16);
  return go(scan2_step_kernel<IO, XT, 1, 64, false>, 64);
}

}  // namespace

hipError_t launch_scan2_step(const Scan2StepArgs& a, bool bf16, hipStream_t stream) {
  if (!a.conv_weight)
    return bf16 ? launch<BF16, BF16>(a, stream) : launch<F32, F32>(a, stream);
  const dim3 grid(static_cast<unsigned>((a.batch * a.conv_dim + kThreads - 1) / kThreads));
  if (bf16) hipLaunchKernelGGL(conv_act_kernel<BF16>, grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL(conv_act_kernel<F32>, grid, dim3(kThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return bf16 ? launch<BF16, F32>(a, stream) : launch<F32, F32>(a, stream);
}

}  // namespace ss
