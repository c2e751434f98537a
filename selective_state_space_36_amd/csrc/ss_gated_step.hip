// ss_gated_step.hip -- one token of the gated linear recurrence, the state advanced in place.
//
// Elementwise: 128 x 5120 bfloat16 with a gate moves 11.8 MB in 4.3 us, one row takes 2.7 us, and
// the call around it 8 us on the host, so nothing is gained below that.
#include "ss_block.h"
#include "ss_gated_math.h"

namespace ss {
namespace {

// V channels of one batch row per thread.
template <class IO, int V, bool GATE>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedStepArgs p, int64_t lanes) {
  using elem = typename IO::elem;
  using L = Lanes<IO, V>;
  using LF = Lanes<F32, V>;
  const int64_t id = blockIdx.x * 256ll + threadIdx.x;
  if (id >= p.batch * lanes) return;
  const int64_t c = id % lanes * V, e = id * V;
  auto io = [&](const void* q) {
    return *reinterpret_cast<const typename L::raw*>(static_cast<const elem*>(q) + e);
  };
  auto f32 = [](const float* q, int64_t at) {
    return *reinterpret_cast<const typename LF::raw*>(q + at);
  };
  const auto r = io(p.r), i = io(p.i), x = io(p.x);
  const auto z = GATE ? io(p.z) : typename L::raw{};
  const auto A = f32(p.A, c), s = f32(p.state, e);
  const auto rb = p.r_bias ? f32(p.r_bias, c) : typename LF::raw{};
  const auto ib = p.i_bias ? f32(p.i_bias, c) : typename LF::raw{};
  float h[V], y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float rg = sigmoid_biased(L::get(r, v), -LF::get(rb, v) * kLog2e);
    const float ig = sigmoid_biased(L::get(i, v), -LF::get(ib, v) * kLog2e);
    const float l = LF::get(A, v) * kLog2e * rg, a = exp2_hw(l);
    h[v] = fmaf(a, LF::get(s, v), decay_scale(l, a) * ig * L::get(x, v));
    y[v] = GATE ? h[v] * silu_f(L::get(z, v)) : h[v];
  }
  *reinterpret_cast<typename LF::raw*>(p.state + e) = LF::put(h);
  *reinterpret_cast<typename L::raw*>(static_cast<elem*>(p.out) + e) = L::put(y);
}

template <class IO, int V>
hipError_t launch(const GatedStepArgs& a, hipStream_t stream) {
  const int64_t lanes = a.d_inner / V;
  const dim3 grid(static_cast<unsigned>((a.batch * lanes + 255) / 256));
  if (a.z)
    hipLaunchKernelGGL((gated_step_kernel<IO, V, true>), grid, dim3(256), 0, stream, a, lanes);
  else
    hipLaunchKernelGGL((gated_step_kernel<IO, V, false>), grid, dim3(256), 0, stream, a, lanes);
  return hipGetLastError();
}

// Two channels per thread where rows and pointers are aligned to them.
template <class IO>
bool pairs(const GatedStepArgs& a) {
  const void* io[] = {a.x, a.r, a.i, a.z, a.out};
  const void* f32[] = {a.state, a.A, a.r_bias, a.i_bias};
  uintptr_t b = 0, f = 0;
  for (const void* q : io) b |= reinterpret_cast<uintptr_t>(q);
  for (const void* q : f32) f |= reinterpret_cast<uintptr_t>(q);
  return a.d_inner % 2 == 0 && b % (2 * sizeof(typename IO::elem)) == 0 && f % 8 == 0;
}

}  // namespace

hipError_t launch_gated_step(const GatedStepArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) return pairs<BF16>(a) ? launch<BF16, 2>(a, stream) : launch<BF16, 1>(a, stream);
  return pairs<F32>(a) ? launch<F32, 2>(a, stream) : launch<F32, 1>(a, stream);
}

}  // namespace ss
