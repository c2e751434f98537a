// ss_head.h -- launch interface between the C-ABI layer (ss_head_api.hip) and the kernels of the
// block around the multi-head scan: its one-token form, its gradients, the RMS norm with the
// residual add, the gated norm and dropout.  Arguments are validated before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ss_block.h"
#include "ss_scan.h"

namespace ss {

// Dropout: elements whose 16 random bits are below `cut` are 0, the others times `up`.
struct DropArgs {
  const uint64_t* rng;     // seed, offset; nullptr: nothing is dropped
  uint32_t cut;
  float up;
};

struct RmsArgs {
  const void* x;           // io; backward: nullptr when neither scale nor branch norm needs it
  const float* residual;   // nullptr: 0
  const float* weight;     // nullptr: 1
  const float* scale;      // nullptr: 1
  bool branch;             // x is normalised before it is scaled
  DropArgs drop;
  float eps;
  void* out;
  float* sum;              // nullptr: not written
  float* rstd;             // nullptr: not written
  float* branch_rstd;      // nullptr: not written
  // backward
  const void* dout;
  const void* s;           // what was normalised: float32 or (s_f32 false) io
  bool s_f32;
  const float* rstd_in;
  const float* branch_rstd_in;
  const float* dsum;
  void* dx;                // nullptr: not written
  float* dresidual;        // nullptr: not written
  float* dweight;          // nullptr: not written
  float* dscale;           // nullptr: not written
  float* workspace;
  int64_t rows, dim;
};

struct GatedNormArgs {
  const void* x;
  const void* z;           // nullptr: no gate
  int64_t z_stride;        // elements from one row of z to the next
  const float* weight;     // nullptr: 1
  bool gate_first;
  float eps;
  void* out;
  float* rstd;             // (rows, groups); nullptr: not written
  // backward
  const void* dout;
  const float* rstd_in;
  void* dx;
  void* dz;
  float* dweight;          // nullptr: not written
  float* workspace;
  int64_t rows, dim, groups;
};

size_t rms_bwd_ws_bytes(int64_t rows, int64_t dim);
hipError_t launch_rms_fwd(const RmsArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_rms_bwd(const RmsArgs& a, bool bf16, hipStream_t stream);
size_t gated_norm_bwd_ws_bytes(int64_t rows, int64_t dim, int64_t groups);
hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, bool bf16, hipStream_t stream);

// One token of the multi-head scan.  x, B and C are rows of the io dtype or, with a convolution
// (conv_weight), parts of the float32 rows `act` that its kernel writes.
struct Scan2StepArgs {
  float* state;            // (batch, nheads, d_state, headdim), in place
  const void* x;
  const void* dt;
  const void* z;           // nullptr: no gate
  const void* B;
  const void* C;
  int64_t x_stride, dt_stride, z_stride, b_stride, c_stride;  // elements between batch rows
  const float* A;
  const float* D;          // nullptr: 0
  const float* dt_bias;    // nullptr: 0
  void* out;
  // convolution (conv_weight nullptr: none)
  void* conv_state;
  const void* xbc;
  int64_t xbc_stride, conv_dim;
  const float* conv_weight;
  const float* conv_bias;
  float* act;
  int32_t conv_k;
  int32_t softplus, headdim, d_state;
  int64_t batch, nheads, ngroups;
  int64_t n_pblk;          // set by the launch
};
hipError_t launch_scan2_step(const Scan2StepArgs& a, bool bf16, hipStream_t stream);

// Gradients of the multi-head scan.
constexpr int kScan2BwdChunk = 64;
constexpr int64_t kScan2BwdMaxWalks = 0xffffffffll / 512;  // (a launch counts threads in 32 bits)
struct Scan2BwdArgs {
  const void* x;
  const void* dt;
  const void* z;           // nullptr: no gate
  const void* B;
  const void* C;
  const void* dout;
  const float* A;
  const float* D;          // nullptr: 0
  const float* dt_bias;    // nullptr: 0
  const float* h0;         // nullptr: zeros
  const float* dh_last;    // nullptr: zeros
  void* dx;
  void* ddt;
  void* dz;
  void* dB;
  void* dC;
  float* dA;
  float* dD;               // nullptr: not written
  float* ddt_bias;         // nullptr: not written
  float* dh0;              // nullptr: not written
  int64_t batch, seqlen, nheads, ngroups;
  int32_t headdim, d_state, softplus;
  // the workspace's parts and the launch's cuts (scan2_bwd_ws_floats sets them)
  float* states;           // (batch, nheads, n_chunks, d_state, headdim): before each chunk
  float* lam;              // the same shape: the adjoint of the state behind each chunk
  float* head_part;        // (batch, n_chunks, 3, nheads): dA, dD, ddt_bias
  float* bc_part;          // (splits, 2, batch, seqlen, ngroups, d_state): dB, dC
  float* decay;            // (2, batch, nheads, n_chunks): of a chunk, where the walks are cut
  int64_t n_chunks, n_pblk, splits;
  bool cut;                // the walks are cut into chunks and joined by launch_scan2_join
};
// Floats of the workspace; with `a` its parts in `ws` are set.
int64_t scan2_bwd_ws_floats(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                            int64_t ngroups, int64_t d_state, Scan2BwdArgs* a, float* ws);
hipError_t launch_scan2_bwd(const Scan2BwdArgs& a, bool bf16, hipStream_t stream);

// Joins walks that were cut: every slot of `states` and `lam` holds the chunk's own part and takes the
// state before it, or the adjoint behind it; `tiled`: in the layout of ss_scan2_bwd_mfma.hip.
// Writes dh0.
hipError_t launch_scan2_join(const Scan2BwdArgs& a, bool tiled, hipStream_t stream);

// Its first two launches with bf16 matrix products (ss_scan2_bwd_mfma.hip): bf16 io, headdim 64,
// d_state 64 or 128, 16-byte aligned arrays.
bool scan2_bwd_mfma_supported(const Scan2BwdArgs& a, bool bf16);
hipError_t launch_scan2_bwd_mfma(const Scan2BwdArgs& a, hipStream_t stream);

hipError_t launch_dropout(const void* x, void* out, const DropArgs& d, int64_t rows, int64_t dim,
                          bool bf16, hipStream_t stream);

}  // namespace ss
