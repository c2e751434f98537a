// ss_gated_step.hip -- one token of the gated linear recurrence, the state advanced in place.
#include "ss_block.h"
#include "ss_gated_math.h"

namespace ss {
namespace {

template <class IO>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedStepArgs p) {
  using elem = typename IO::elem;
  const int64_t e = blockIdx.x * 256ll + threadIdx.x;
  if (e >= p.batch * p.d_inner) return;
  const int64_t d = e % p.d_inner;
  const float rg = sigmoid_f(IO::load(static_cast<const elem*>(p.r), e) +
                             (p.r_bias ? p.r_bias[d] : 0.0f));
  const float ig = sigmoid_f(IO::load(static_cast<const elem*>(p.i), e) +
                             (p.i_bias ? p.i_bias[d] : 0.0f));
  const Decay k = decay_f(p.A[d] * rg);
  const float h = fmaf(k.a, p.state[e], k.s * ig * IO::load(static_cast<const elem*>(p.x), e));
  p.state[e] = h;
  const float y = p.z ? h * silu_f(IO::load(static_cast<const elem*>(p.z), e)) : h;
  static_cast<elem*>(p.out)[e] = IO::from_float(y);
}

}  // namespace

hipError_t launch_gated_step(const GatedStepArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.batch * a.d_inner + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL((gated_step_kernel<BF16>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((gated_step_kernel<F32>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace ss
