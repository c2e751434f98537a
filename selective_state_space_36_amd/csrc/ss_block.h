// ss_block.h -- launch interface between the C-ABI layer (ss_block_api.hip) and the kernels of
// the recurrent block's operators: the gated linear recurrence, the layer norm and the causal
// convolution.  Arguments are validated before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ss_scan.h"

namespace ss {

struct GatedArgs {
  const void* x;
  const void* r;
  const void* i;
  const void* z;           // nullptr: no output gate
  const float* A;
  const float* r_bias;     // nullptr: 0
  const float* i_bias;     // nullptr: 0
  const uint8_t* starts;   // nullptr: none
  const float* h0;         // nullptr: zeros
  float* h_last;           // nullptr: not written
  void* out;
  float* states;           // nullptr: not written (forward); chunk-end states (backward)
  // backward
  const void* dout;
  const float* dh_last;    // nullptr: 0
  void* dx;
  void* dr;
  void* di;
  void* dz;
  float* dA;
  float* dr_bias;          // nullptr: not written
  float* di_bias;          // nullptr: not written
  float* dh0;              // nullptr: not written
  void* workspace;
  int64_t batch, seqlen, d_inner;
  int64_t n_chunks;        // ceil(seqlen / SS_GATED_CHUNK)
};

// Steps of a wave, and of a workgroup's tile, of the forward; steps of a wave of the backward,
// whose tile is SS_GATED_CHUNK.
constexpr int kGatedFwdSteps = 16, kGatedFwdTile = 128, kGatedBwdSteps = 8;
size_t gated_fwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner);
size_t gated_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, bool states_given);
hipError_t launch_gated_fwd(const GatedArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_gated_bwd(const GatedArgs& a, bool bf16, hipStream_t stream);

struct GatedStepArgs {
  float* state;
  const void* x;
  const void* r;
  const void* i;
  const void* z;
  const float* A;
  const float* r_bias;
  const float* i_bias;
  void* out;
  int64_t batch, d_inner;
};
hipError_t launch_gated_step(const GatedStepArgs& a, bool bf16, hipStream_t stream);

struct NormArgs {
  const void* x;           // forward: x; backward: s
  const float* residual;
  const float* weight;
  const float* bias;
  float eps;
  void* out;
  float* sum;
  float* mean;
  float* rstd;
  // backward
  const void* dout;
  const float* mean_in;
  const float* rstd_in;
  const float* dsum;
  void* dx;
  float* dresidual;
  float* dweight;
  float* dbias;
  void* workspace;
  bool s_f32;              // backward: s is float32 whatever the io dtype
  int64_t rows, dim;
};
size_t norm_bwd_ws_bytes(int64_t rows, int64_t dim);
hipError_t launch_norm_fwd(const NormArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs& a, bool bf16, hipStream_t stream);

struct ConvArgs {
  const void* x;
  const float* weight;
  const float* bias;
  const void* x_prev;
  const uint8_t* starts;
  void* out;
  void* conv_state;        // one-token form
  // backward
  const void* dout;
  void* dx;
  float* dweight;
  float* dbias;
  void* dx_prev;
  void* workspace;
  int64_t batch, seqlen, d_inner;
  int32_t k;
  int32_t silu;
};
size_t conv_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, int32_t k);
hipError_t launch_conv_fwd(const ConvArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs& a, bool bf16, hipStream_t stream);

// Fills and copies for empty problems (kernels, so that they can be captured into a graph).
hipError_t launch_zero(float* p, int64_t n, hipStream_t stream);
hipError_t launch_zero_bytes(void* p, int64_t bytes, hipStream_t stream);
hipError_t launch_copy(float* dst, const float* src, int64_t n, hipStream_t stream);

// Sums over the lines of partial results, for up to five outputs of `cols` values:
// out[c * out_stride] = sum over r < lines of src[r * stride + c], in a fixed order.
struct ColumnSums {
  struct Job {
    const float* src;
    float* out;
    int64_t out_stride;
  };
  Job job[5];
  int32_t jobs;
  int64_t lines, stride, cols;
  // Adds an output; a null one is not wanted.
  void add(const float* src, float* out, int64_t out_stride) {
    if (out) job[jobs++] = Job{src, out, out_stride};
  }
};
hipError_t launch_column_sums(const ColumnSums& p, hipStream_t stream);

// Calls f with the truth values as compile-time constants.
template <class F>
void with_bools(F f, bool a, bool b) {
  using std::bool_constant;
  if (a)
    b ? f(bool_constant<true>{}, bool_constant<true>{})
      : f(bool_constant<true>{}, bool_constant<false>{});
  else
    b ? f(bool_constant<false>{}, bool_constant<true>{})
      : f(bool_constant<false>{}, bool_constant<false>{});
}

}  // namespace ss
