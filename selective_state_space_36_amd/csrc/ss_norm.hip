// ss_norm.hip -- layer norm over the last axis with the residual add, and its gradients.
#include "ss_block.h"
#include "ss_device.h"

namespace ss {
namespace {

constexpr int kThreads = 256;

// Sum over the workgroup, the same in every lane.
__device__ float block_sum(float v, float* lds) {
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < kThreads / 64; ++w) s += lds[w];
  return s;
}

// One workgroup per row, three passes over it.
template <class IO>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(NormArgs p) {
  using elem = typename IO::elem;
  __shared__ float lds[kThreads / 64];
  const int64_t row = blockIdx.x, at = row * p.dim;
  auto value = [&](int64_t c) {
    const float x = IO::load(static_cast<const elem*>(p.x), at + c);
    return p.residual ? x + p.residual[at + c] : x;
  };
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) s += value(c);
  const float mu = block_sum(s, lds) / static_cast<float>(p.dim);
  float v = 0.0f;
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
    const float t = value(c) - mu;
    v = fmaf(t, t, v);
  }
  const float var = block_sum(v, lds) / static_cast<float>(p.dim);
  const float rstd = 1.0f / __builtin_sqrtf(var + p.eps);
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
    const float t = value(c);
    const float xh = (t - mu) * rstd;
    const float w = p.weight ? p.weight[c] : 1.0f, b = p.bias ? p.bias[c] : 0.0f;
    static_cast<elem*>(p.out)[at + c] = IO::from_float(fmaf(xh, w, b));
    if (p.sum) p.sum[at + c] = t;
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

template <class IO, class S>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormArgs p) {
  using elem = typename IO::elem;
  __shared__ float lds[kThreads / 64];
  const int64_t row = blockIdx.x, at = row * p.dim;
  const float mu = p.mean_in[row], rstd = p.rstd_in[row];
  const auto* sp = static_cast<const typename S::elem*>(p.x);
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
    const float xh = (S::load(sp, at + c) - mu) * rstd;
    const float g = IO::load(static_cast<const elem*>(p.dout), at + c) *
                    (p.weight ? p.weight[c] : 1.0f);
    s1 += g;
    s2 = fmaf(g, xh, s2);
  }
  const float c1 = block_sum(s1, lds) / static_cast<float>(p.dim);
  const float c2 = block_sum(s2, lds) / static_cast<float>(p.dim);
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
    const float xh = (S::load(sp, at + c) - mu) * rstd;
    const float g = IO::load(static_cast<const elem*>(p.dout), at + c) *
                    (p.weight ? p.weight[c] : 1.0f);
    float ds = rstd * (g - c1 - xh * c2);
    if (p.dsum) ds += p.dsum[at + c];
    if (p.dx) static_cast<elem*>(p.dx)[at + c] = IO::from_float(ds);
    if (p.dresidual) p.dresidual[at + c] = ds;
  }
}

// One thread per column over all rows.
template <class IO, class S>
__global__ __launch_bounds__(64) void norm_param_kernel(NormArgs p) {
  using elem = typename IO::elem;
  const int64_t c = blockIdx.x * 64ll + threadIdx.x;
  if (c >= p.dim) return;
  const auto* sp = static_cast<const typename S::elem*>(p.x);
  float w = 0.0f, b = 0.0f;
  for (int64_t row = 0; row < p.rows; ++row) {
    const float dy = IO::load(static_cast<const elem*>(p.dout), row * p.dim + c);
    w = fmaf(dy, (S::load(sp, row * p.dim + c) - p.mean_in[row]) * p.rstd_in[row], w);
    b += dy;
  }
  if (p.dweight) p.dweight[c] = w;
  if (p.dbias) p.dbias[c] = b;
}

template <class IO, class S>
hipError_t launch_bwd(const NormArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((norm_bwd_kernel<IO, S>), dim3(static_cast<unsigned>(a.rows)),
                     dim3(kThreads), 0, stream, a);
  if (a.dweight || a.dbias)
    hipLaunchKernelGGL((norm_param_kernel<IO, S>),
                       dim3(static_cast<unsigned>((a.dim + 63) / 64)), dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t norm_bwd_ws_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_norm_fwd(const NormArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.rows));
  if (bf16)
    hipLaunchKernelGGL((norm_fwd_kernel<BF16>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((norm_fwd_kernel<F32>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, bool bf16, hipStream_t stream) {
  if (!bf16) return launch_bwd<F32, F32>(a, stream);
  return a.s_f32 ? launch_bwd<BF16, F32>(a, stream) : launch_bwd<BF16, BF16>(a, stream);
}

}  // namespace ss
