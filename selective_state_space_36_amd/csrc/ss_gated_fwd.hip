// ss_gated_fwd.hip -- the gated linear recurrence over a whole sequence.
#include "ss_block.h"
#include "ss_gated_math.h"

namespace ss {
namespace {

// One thread per channel, one step after the other.
template <class IO>
__global__ __launch_bounds__(64) void gated_fwd_kernel(GatedArgs p) {
  using elem = typename IO::elem;
  const int64_t ch = blockIdx.x * 64ll + threadIdx.x;
  if (ch >= p.batch * p.d_inner) return;
  const int64_t b = ch / p.d_inner, d = ch % p.d_inner;
  const float A = p.A[d], rb = p.r_bias ? p.r_bias[d] : 0.0f, ib = p.i_bias ? p.i_bias[d] : 0.0f;
  float h = p.h0 ? p.h0[ch] : 0.0f;
  for (int64_t t = 0; t < p.seqlen; ++t) {
    const int64_t e = (b * p.seqlen + t) * p.d_inner + d;
    const float rg = sigmoid_f(IO::load(static_cast<const elem*>(p.r), e) + rb);
    const float ig = sigmoid_f(IO::load(static_cast<const elem*>(p.i), e) + ib);
    const Decay k = decay_f(A * rg);
    const float in = k.s * ig * IO::load(static_cast<const elem*>(p.x), e);
    const bool fresh = p.starts && p.starts[b * p.seqlen + t];
    h = fresh ? in : fmaf(k.a, h, in);
    if (p.out) {
      const float y = p.z ? h * silu_f(IO::load(static_cast<const elem*>(p.z), e)) : h;
      static_cast<elem*>(p.out)[e] = IO::from_float(y);
    }
    if (p.states && ((t + 1) % SS_GATED_CHUNK == 0 || t + 1 == p.seqlen))
      p.states[(b * p.n_chunks + t / SS_GATED_CHUNK) * p.d_inner + d] = h;
  }
  if (p.h_last) p.h_last[ch] = h;
}

}  // namespace

size_t gated_fwd_ws_bytes(int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_gated_fwd(const GatedArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.batch * a.d_inner + 63) / 64));
  if (bf16)
    hipLaunchKernelGGL((gated_fwd_kernel<BF16>), grid, dim3(64), 0, stream, a);
  else
    hipLaunchKernelGGL((gated_fwd_kernel<F32>), grid, dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace ss
