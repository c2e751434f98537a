// ss_conv.hip -- the causal depthwise convolution, its gradients and its one-token form.
#include "ss_block.h"
#include "ss_gated_math.h"

namespace ss {
namespace {

// x at step t of row b (t may be negative: the window before the sequence).
template <class IO>
__device__ __forceinline__ float tap(const ConvArgs& p, int64_t b, int64_t t, int64_t d) {
  using elem = typename IO::elem;
  if (t >= 0) return IO::load(static_cast<const elem*>(p.x), (b * p.seqlen + t) * p.d_inner + d);
  return p.x_prev ? IO::load(static_cast<const elem*>(p.x_prev),
                             (b * (p.k - 1) + p.k - 1 + t) * p.d_inner + d)
                  : 0.0f;
}

__device__ __forceinline__ bool fresh(const ConvArgs& p, int64_t b, int64_t t) {
  return p.starts && p.starts[b * p.seqlen + t];
}

template <class IO>
__device__ float preact(const ConvArgs& p, int64_t b, int64_t t, int64_t d) {
  int far = 0;  // the oldest tap in the same sequence
  while (far < p.k - 1 && !(t - far >= 0 && fresh(p, b, t - far))) ++far;
  float acc = p.bias ? p.bias[d] : 0.0f;
  for (int lag = far; lag >= 0; --lag)
    acc = fmaf(p.weight[d * p.k + p.k - 1 - lag], tap<IO>(p, b, t - lag, d), acc);
  return acc;
}

template <class IO>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs p) {
  const int64_t e = blockIdx.x * 256ll + threadIdx.x;
  if (e >= p.batch * p.seqlen * p.d_inner) return;
  const int64_t d = e % p.d_inner, bt = e / p.d_inner;
  const float v = preact<IO>(p, bt / p.seqlen, bt % p.seqlen, d);
  static_cast<typename IO::elem*>(p.out)[e] = IO::from_float(p.silu ? silu_f(v) : v);
}

template <class IO>
__device__ float pre_grad(const ConvArgs& p, int64_t b, int64_t t, int64_t d) {
  float g = IO::load(static_cast<const typename IO::elem*>(p.dout),
                     (b * p.seqlen + t) * p.d_inner + d);
  if (p.silu) {
    const float v = preact<IO>(p, b, t, d);
    const float sg = sigmoid_f(v);
    g *= sg * fmaf(v, 1.0f - sg, 1.0f);
  }
  return g;
}

// dx (and dx_prev for t < 0), one thread per element.
template <class IO>
__global__ __launch_bounds__(256) void conv_dx_kernel(ConvArgs p) {
  const int64_t e = blockIdx.x * 256ll + threadIdx.x;
  const int64_t steps = p.seqlen + p.k - 1;
  if (e >= p.batch * steps * p.d_inner) return;
  const int64_t d = e % p.d_inner, bt = e / p.d_inner;
  const int64_t b = bt / steps, t = bt % steps - (p.k - 1);
  if (t < 0 && !p.dx_prev) return;
  float acc = 0.0f;
  for (int lag = 0; lag < p.k && t + lag < p.seqlen; ++lag) {
    if (t + lag < 0) continue;
    if (lag > 0 && fresh(p, b, t + lag)) break;  // a start between t and t + lag cuts the tap
    acc = fmaf(p.weight[d * p.k + p.k - 1 - lag], pre_grad<IO>(p, b, t + lag, d), acc);
  }
  using elem = typename IO::elem;
  if (t >= 0)
    static_cast<elem*>(p.dx)[(b * p.seqlen + t) * p.d_inner + d] = IO::from_float(acc);
  else
    static_cast<elem*>(p.dx_prev)[(b * (p.k - 1) + p.k - 1 + t) * p.d_inner + d] =
        IO::from_float(acc);
}

// dweight and dbias, one thread per channel over all tokens.
template <class IO>
__global__ __launch_bounds__(64) void conv_dw_kernel(ConvArgs p) {
  const int64_t d = blockIdx.x * 64ll + threadIdx.x;
  if (d >= p.d_inner) return;
  float w[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s = 0.0f;
  for (int64_t b = 0; b < p.batch; ++b)
    for (int64_t t = 0; t < p.seqlen; ++t) {
      const float g = pre_grad<IO>(p, b, t, d);
      s += g;
      for (int lag = 0; lag < p.k; ++lag) {
        w[lag] = fmaf(g, tap<IO>(p, b, t - lag, d), w[lag]);
        if (t - lag < 0 ? false : fresh(p, b, t - lag)) break;
      }
    }
  for (int lag = 0; lag < p.k; ++lag) p.dweight[d * p.k + p.k - 1 - lag] = w[lag];
  if (p.dbias) p.dbias[d] = s;
}

template <class IO>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs p) {
  using elem = typename IO::elem;
  const int64_t e = blockIdx.x * 256ll + threadIdx.x;
  if (e >= p.batch * p.d_inner) return;
  const int64_t b = e / p.d_inner, d = e % p.d_inner;
  elem* st = static_cast<elem*>(p.conv_state) + b * (p.k - 1) * p.d_inner + d;
  const elem xv = static_cast<const elem*>(p.x)[e];
  float acc = p.bias ? p.bias[d] : 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const elem v = j < p.k - 1 ? st[j * p.d_inner] : xv;
    acc = fmaf(p.weight[d * p.k + j], IO::widen(v), acc);
    if (j > 0) st[(j - 1) * p.d_inner] = v;
  }
  static_cast<elem*>(p.out)[e] = IO::from_float(p.silu ? silu_f(acc) : acc);
}

dim3 blocks(int64_t n, int per) { return dim3(static_cast<unsigned>((n + per - 1) / per)); }

}  // namespace

size_t conv_bwd_ws_bytes(int64_t, int64_t, int64_t, int32_t, bool) { return 0; }

hipError_t launch_conv_fwd(const ConvArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid = blocks(a.batch * a.seqlen * a.d_inner, 256);
  if (bf16)
    hipLaunchKernelGGL((conv_fwd_kernel<BF16>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((conv_fwd_kernel<F32>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_conv_bwd(const ConvArgs& a, bool bf16, hipStream_t stream) {
  const dim3 gx = blocks(a.batch * (a.seqlen + a.k - 1) * a.d_inner, 256);
  const dim3 gw = blocks(a.d_inner, 64);
  if (bf16) {
    hipLaunchKernelGGL((conv_dx_kernel<BF16>), gx, dim3(256), 0, stream, a);
    hipLaunchKernelGGL((conv_dw_kernel<BF16>), gw, dim3(64), 0, stream, a);
  } else {
    hipLaunchKernelGGL((conv_dx_kernel<F32>), gx, dim3(256), 0, stream, a);
    hipLaunchKernelGGL((conv_dw_kernel<F32>), gw, dim3(64), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_conv_step(const ConvArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid = blocks(a.batch * a.d_inner, 256);
  if (bf16)
    hipLaunchKernelGGL((conv_step_kernel<BF16>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((conv_step_kernel<F32>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace ss
