// ss_gated_bwd.hip -- gradients of the gated linear recurrence.
#include "ss_block.h"
#include "ss_gated_math.h"

namespace ss {
namespace {

constexpr int kC = SS_GATED_CHUNK;

// One thread per channel, the chunks from the last to the first: the chunk's states are run
// forward again from the chunk-end state before it (kept in registers or scratch), then the
// adjoint runs back over it.
template <class IO>
__global__ __launch_bounds__(64) void gated_bwd_kernel(GatedArgs p, const float* states,
                                                       float* part) {
  using elem = typename IO::elem;
  const int64_t ch = blockIdx.x * 64ll + threadIdx.x;
  const int64_t rows = p.batch * p.d_inner;
  if (ch >= rows) return;
  const int64_t b = ch / p.d_inner, d = ch % p.d_inner;
  const float A = p.A[d], rb = p.r_bias ? p.r_bias[d] : 0.0f, ib = p.i_bias ? p.i_bias[d] : 0.0f;
  float carry = p.dh_last ? p.dh_last[ch] : 0.0f;
  float sA = 0.0f, sr = 0.0f, si = 0.0f;
  for (int64_t c = p.n_chunks - 1; c >= 0; --c) {
    const int64_t t0 = c * kC, n = p.seqlen - t0 < kC ? p.seqlen - t0 : kC;
    float hp[kC];  // h_{t-1}
    float h = c ? states[(b * p.n_chunks + c - 1) * p.d_inner + d] : p.h0 ? p.h0[ch] : 0.0f;
    for (int j = 0; j < n; ++j) {
      const int64_t t = t0 + j, e = (b * p.seqlen + t) * p.d_inner + d;
      if (p.starts && p.starts[b * p.seqlen + t]) h = 0.0f;
      hp[j] = h;
      const float rg = sigmoid_f(IO::load(static_cast<const elem*>(p.r), e) + rb);
      const float ig = sigmoid_f(IO::load(static_cast<const elem*>(p.i), e) + ib);
      const Decay k = decay_f(A * rg);
      h = fmaf(k.a, h, k.s * ig * IO::load(static_cast<const elem*>(p.x), e));
    }
    for (int j = static_cast<int>(n) - 1; j >= 0; --j) {
      const int64_t t = t0 + j, e = (b * p.seqlen + t) * p.d_inner + d;
      const float x = IO::load(static_cast<const elem*>(p.x), e);
      const float rg = sigmoid_f(IO::load(static_cast<const elem*>(p.r), e) + rb);
      const float ig = sigmoid_f(IO::load(static_cast<const elem*>(p.i), e) + ib);
      const Decay k = decay_f(A * rg);
      float g = IO::load(static_cast<const elem*>(p.dout), e);
      if (p.z) {
        const float z = IO::load(static_cast<const elem*>(p.z), e);
        const float sg = sigmoid_f(z);
        const float ht = fmaf(k.a, hp[j], k.s * ig * x);
        static_cast<elem*>(p.dz)[e] = IO::from_float(g * ht * (sg * fmaf(z, 1.0f - sg, 1.0f)));
        g *= z * sg;
      }
      const float lam = g + carry;
      const bool fresh = p.starts && p.starts[b * p.seqlen + t];
      carry = fresh ? 0.0f : k.a * lam;
      const float slope = k.s > 0.0f ? k.a * k.a * rcp_hw(k.s) : 0.0f;
      const float dl = lam * (k.a * hp[j] - ig * x * slope);
      const float dr = dl * A * rg * (1.0f - rg);
      const float di = lam * k.s * x * ig * (1.0f - ig);
      static_cast<elem*>(p.dx)[e] = IO::from_float(lam * k.s * ig);
      static_cast<elem*>(p.dr)[e] = IO::from_float(dr);
      static_cast<elem*>(p.di)[e] = IO::from_float(di);
      sA += dl * rg;
      sr += dr;
      si += di;
    }
  }
  if (p.dh0) p.dh0[ch] = carry;
  part[ch] = sA;
  part[rows + ch] = sr;
  part[2 * rows + ch] = si;
}

__global__ __launch_bounds__(64) void gated_reduce_kernel(GatedArgs p, const float* part) {
  const int64_t d = blockIdx.x * 64ll + threadIdx.x;
  if (d >= p.d_inner) return;
  const int64_t rows = p.batch * p.d_inner;
  float s[3] = {0.0f, 0.0f, 0.0f};
  for (int64_t b = 0; b < p.batch; ++b)
    for (int q = 0; q < 3; ++q) s[q] += part[q * rows + b * p.d_inner + d];
  p.dA[d] = s[0];
  if (p.dr_bias) p.dr_bias[d] = s[1];
  if (p.di_bias) p.di_bias[d] = s[2];
}

}  // namespace

size_t gated_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, bool bf16, bool given) {
  const int64_t rows = batch * d_inner, chunks = (seqlen + kC - 1) / kC;
  return static_cast<size_t>(rows) * sizeof(float) * (3 + (given ? 0 : chunks)) + 16 +
         (given ? 0 : gated_fwd_ws_bytes(batch, seqlen, d_inner, bf16));
}

hipError_t launch_gated_bwd(const GatedArgs& a, bool bf16, hipStream_t stream) {
  float* part = static_cast<float*>(a.workspace);
  const float* states = a.states;
  if (!states) {
    GatedArgs f = a;
    f.out = nullptr;
    f.h_last = nullptr;
    f.states = part + 3 * a.batch * a.d_inner;
    states = f.states;
    const uintptr_t end = reinterpret_cast<uintptr_t>(f.states + a.batch * a.n_chunks * a.d_inner);
    f.workspace = reinterpret_cast<void*>((end + 15) / 16 * 16);
    const hipError_t e = launch_gated_fwd(f, bf16, stream);
    if (e != hipSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>((a.batch * a.d_inner + 63) / 64));
  if (bf16)
    hipLaunchKernelGGL((gated_bwd_kernel<BF16>), grid, dim3(64), 0, stream, a, states, part);
  else
    hipLaunchKernelGGL((gated_bwd_kernel<F32>), grid, dim3(64), 0, stream, a, states, part);
  hipLaunchKernelGGL(gated_reduce_kernel, dim3(static_cast<unsigned>((a.d_inner + 63) / 64)),
                     dim3(64), 0, stream, a, part);
  return hipGetLastError();
}

}  // namespace ss
