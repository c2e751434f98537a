/*
 * ss_scan.h -- C ABI of the MI355X (gfx950) selective state-space scan library (libssscan.so).
 *
 * The operation (Mamba's selective SSM, "S6"), for every batch row b and channel d:
 *
 *     dt_t    = softplus(delta[b,t,d] + delta_bias[d])      (or the raw sum, softplus off)
 *     h_t[n]  = exp(dt_t * A[d,n]) * h_{t-1}[n] + dt_t * B[b,t,n] * u[b,t,d]
 *     y_t     = sum_n C[b,t,n] * h_t[n] + D[d] * u[b,t,d]
 *     out     = y_t * silu(z[b,t,d])                        (when z is given)
 *
 * Sources (web pages; cited by title and section):
 *   - "Mamba: Linear-Time Sequence Modeling with Selective State Spaces" reading guide
 *     (xyznot.com): "Método" (continuous SSM, ZOH discretisation Abar = exp(dt A), the
 *     recurrence and y_t = C h_t), "O Mecanismo de Seleção (S6)" (B_t, C_t and dt_t depend on the
 *     input; dt = softplus(Parameter + s(x))), "Expansão de Estado Ciente de Hardware" (the
 *     (batch, L, d_inner, d_state) state is never written to HBM; the output is contracted with C
 *     first), "Perguntas" (decode keeps a fixed d_inner x d_state state per layer, O(1) per token).
 *   - "O que é um modelo Mamba?" (ibm.com): the output equation with the D term, the diagonal A,
 *     and the Mamba block in which the SSM output is multiplied by the activated gate z.
 *   - "Как работает Mamba" (aivaro.ru), section 3 "Selective Scan": the function shape
 *     selective_scan(u, delta, A, B, C, D) with u, delta [batch, length, d_in] and B, C
 *     [batch, length, d_state], and the first-order input term B_bar = delta * B.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers owned by the caller; arrays are contiguous and row-major.
 *     The library allocates no device memory and keeps no state between calls (the one
 *     exception: the static scratch array of ss_scan_fwd_noalloc, described there).
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Calls only enqueue
 *     work and return; they never synchronise, print or throw.
 *   - Argument errors are detected before anything is launched and leave all outputs untouched.
 *     A launch failure is reported as SS_ERR_HIP.  ss_last_error() gives a thread-local message.
 *   - All index arithmetic is 64-bit.  Calls are thread-safe.
 *   - Element types: SS_F32 (float) or SS_BF16 (bfloat16 bits) for u, delta, z, B, C and out;
 *     A, D, delta_bias, the state, h0 and h_last are always float32.  Arithmetic and the state
 *     are float32; out is rounded to its dtype with round-to-nearest-even.
 */
#ifndef SS_SCAN_H
#define SS_SCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SS_OK = 0,
  SS_ERR_INVALID_ARG = 1, /* NULL required pointer, negative or inconsistent size, aliasing */
  SS_ERR_UNSUPPORTED = 2, /* d_state outside 1..64, unknown dtype or flag, misaligned element */
  SS_ERR_HIP = 3          /* the HIP runtime reported an error while launching */
} ss_status;

typedef enum { SS_F32 = 0, SS_BF16 = 1 } ss_dtype;

/*
 * Option bits (an entry point given a bit it does not take -> SS_ERR_UNSUPPORTED).
 *   SS_FLAG_ZOH_EXACT (prefill and decode): the input term uses the exact zero-order-hold
 *     discretisation of the continuous system (reading guide, "Método": B_bar =
 *     (dt A)^-1 (exp(dt A) - I) dt B, which for the diagonal A is B_bar[n] =
 *     (exp(dt A[d,n]) - 1) / A[d,n] * B[n], and dt * B[n] where A[d,n] == 0) in place of the
 *     first-order dt * B[n] of the default (aivaro.ru, section 3).  A_bar = exp(dt A) either
 *     way.  It costs a few more operations per state update.
 *   SS_FLAG_STATES_GIVEN (ss_scan_bwd only): the workspace already begins with the chunk-end
 *     states of these inputs, as written by ss_scan_fwd_states; the backward then skips its own
 *     forward pass.
 */
enum { SS_FLAG_ZOH_EXACT = 1, SS_FLAG_STATES_GIVEN = 2 };

/*
 * Prefill: the whole sequence in one call.
 *
 *   u, delta, z, out : (batch, seqlen, d_inner), io dtype.  z == NULL: no gate.
 *   B, C             : (batch, seqlen, d_state), io dtype, shared by all channels.
 *   A                : (d_inner, d_state) float32, the diagonal of each channel's A.
 *   D                : (d_inner) float32, skip weight; NULL means 0.
 *   delta_bias       : (d_inner) float32, added to delta before softplus; NULL means 0.
 *   delta_softplus   : nonzero -> dt = softplus(delta + bias); zero -> dt = delta + bias.
 *   h0               : (batch, d_inner, d_state) float32 initial state; NULL means zeros.
 *   h_last           : (batch, d_inner, d_state) float32 final state, written if non-NULL.
 *   workspace        : optional device scratch for splitting long sequences in time.  Size it
 *                      with ss_scan_fwd_workspace_bytes(); with less (or NULL/0) the library
 *                      splits less (or not at all): the result is the same up to rounding,
 *                      only slower on shapes with few channels.
 * out and h_last must not overlap any input or each other (SS_ERR_INVALID_ARG).
 * d_state outside 1..64, d_inner above 2^24 or seqlen above 2^31 - 1 -> SS_ERR_UNSUPPORTED.
 * batch == 0, seqlen == 0 or d_inner == 0 is a no-op returning SS_OK (with seqlen == 0 and
 * h_last given, h_last receives h0, or zeros).
 */
ss_status ss_scan_fwd(const void* u, const void* delta, const float* A, const void* B,
                      const void* C, const float* D, const void* z, const float* delta_bias,
                      int delta_softplus, const float* h0, float* h_last, void* out,
                      int64_t batch, int64_t seqlen, int64_t d_inner, int64_t d_state,
                      ss_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes ss_scan_fwd can use for this shape (0 when it would not split in time). */
size_t ss_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                   int64_t d_state, ss_dtype dtype);

/*
 * Prefill that allocates nothing, for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation.  The same operation,
 * arguments and results as ss_scan_fwd, without the workspace: when the automatic time split
 * is used (shapes with few channels and long sequences), its segment end states and step sums
 * live in a static device array of SS_NOALLOC_SCRATCH_BYTES bytes inside the library, one per
 * GPU, held from its first use on that GPU until the process ends.
 *   - The array of the calling thread's current device is used; `stream` must belong to that
 *     device.  Its address is looked up once per device (hipGetSymbolAddress) and cached.
 *   - Every call on one GPU shares that GPU's array: calls that overlap in time on one GPU (on
 *     different streams, or from several threads) race on it and give wrong results.  Calls
 *     ordered on one stream are safe; nothing in the array needs to start at zero.
 *   - 8 MiB holds the automatic split of every shape with d_state <= 16 on a 256-CU MI355X
 *     (the split targets about 24 waves per SIMD with 4 channels per wave, so its carries stay
 *     below 98304 rows of d_state + 1 floats, 6.7 MB).  A shape whose split needs more (d_state
 *     above 16 with few channels and long sequences) -> SS_ERR_INVALID_ARG before any launch;
 *     ss_scan_fwd with a workspace takes every shape.
 *   - No hipMalloc, hipFree or other allocating call is made.
 */
#define SS_NOALLOC_SCRATCH_BYTES (8u << 20)
ss_status ss_scan_fwd_noalloc(const void* u, const void* delta, const float* A, const void* B,
                              const void* C, const float* D, const void* z,
                              const float* delta_bias, int delta_softplus, const float* h0,
                              float* h_last, void* out, int64_t batch, int64_t seqlen,
                              int64_t d_inner, int64_t d_state, ss_dtype dtype, void* stream);

/*
 * Prefill with an explicit time split and options.  nseg > 0 forces the sequence to be cut into
 * that many segments (each scanned from a carried state; the carries come from a first summary
 * pass over the segments, the blockwise associative decomposition of the recurrence); nseg == 0
 * chooses automatically.  Used to check that the result does not depend on the split.  With
 * nseg > 1 the workspace must hold ss_scan_fwd_ex_workspace_bytes(..., nseg) bytes
 * (SS_ERR_INVALID_ARG otherwise).  flags: SS_FLAG_* bits (0 = the ss_scan_fwd operation).
 */
ss_status ss_scan_fwd_ex(const void* u, const void* delta, const float* A, const void* B,
                         const void* C, const float* D, const void* z, const float* delta_bias,
                         int delta_softplus, const float* h0, float* h_last, void* out,
                         int64_t batch, int64_t seqlen, int64_t d_inner, int64_t d_state,
                         ss_dtype dtype, void* workspace, size_t workspace_bytes, int32_t nseg,
                         uint32_t flags, void* stream);

size_t ss_scan_fwd_ex_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                      int64_t d_state, ss_dtype dtype, int32_t nseg);

/*
 * Prefill that also saves the state after every 16-step chunk, for a later backward (the
 * reading guide, "Expansão de Estado Ciente de Hardware", keeps intermediate states out of
 * memory and recomputes them in the backward pass; the chunk-end states are the points the
 * recomputation restarts from).  As ss_scan_fwd (first-order input term), plus:
 *   states : (batch, ceil(seqlen / 16), d_inner, d_state) float32, written: states[b,c,d,:] is
 *            the state after step min(16 c + 15, seqlen - 1).  Caller-owned, of
 *            ss_scan_fwd_states_bytes() bytes; it must not overlap the inputs, out, h_last or
 *            the workspace.  It is exactly the first part of the workspace
 *            ss_scan_bwd takes with SS_FLAG_STATES_GIVEN: a training step points `states` at the
 *            start of a buffer of ss_scan_bwd_workspace_bytes() bytes and passes that buffer to
 *            the backward.
 */
ss_status ss_scan_fwd_states(const void* u, const void* delta, const float* A, const void* B,
                             const void* C, const float* D, const void* z,
                             const float* delta_bias, int delta_softplus, const float* h0,
                             float* h_last, void* out, float* states, int64_t batch,
                             int64_t seqlen, int64_t d_inner, int64_t d_state, ss_dtype dtype,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of the states ss_scan_fwd_states writes for this shape (0 for an empty problem). */
size_t ss_scan_fwd_states_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                int64_t d_state);

/*
 * Prefill with the block's front end fused in: instead of u the call takes the block's x and
 * forms the SSM input itself (IBM explainer, Mamba-block walk-through: x_proj passes a
 * one-dimensional convolution, then SiLU, and the result feeds the SSM):
 *
 *     u[b,t,d] = silu( conv_bias[d] + sum_{j<conv_k} conv_weight[d,j] * x[b, t-conv_k+1+j, d] )
 *
 * a causal (step t sees x up to t), depthwise (one kernel per channel) convolution of width
 * conv_k in 1..4 (the pages give no width; 4 is the usual choice).  u is kept in float32 and
 * never written to memory.  Everything else is ss_scan_fwd_ex with u replaced by:
 *   x            : (batch, seqlen, d_inner), io dtype.
 *   conv_weight  : (d_inner, conv_k) float32, required.
 *   conv_bias    : (d_inner) float32; NULL means 0.
 *   x_prev       : (batch, conv_k - 1, d_inner), io dtype: the conv_k - 1 inputs that came
 *                  before t = 0 (oldest first), e.g. the end of the previous call's x; NULL
 *                  means zeros.
 * conv_k outside 1..4 -> SS_ERR_UNSUPPORTED; conv_weight NULL -> SS_ERR_INVALID_ARG.
 */
ss_status ss_scan_fwd_conv(const void* x, const float* conv_weight, const float* conv_bias,
                           const void* x_prev, int32_t conv_k, const void* delta, const float* A,
                           const void* B, const void* C, const float* D, const void* z,
                           const float* delta_bias, int delta_softplus, const float* h0,
                           float* h_last, void* out, int64_t batch, int64_t seqlen,
                           int64_t d_inner, int64_t d_state, ss_dtype dtype, void* workspace,
                           size_t workspace_bytes, int32_t nseg, uint32_t flags, void* stream);

/*
 * Decode: advance a resident state by ONE token (the recurrence above for a single t).
 *
 *   state        : (batch, d_inner, d_state) float32, read and overwritten IN PLACE.
 *   u, delta, z  : (batch, d_inner), io dtype; z == NULL: no gate.
 *   B, C         : (batch, d_state), io dtype.
 *   out          : (batch, d_inner), io dtype.
 *   A, D, delta_bias, delta_softplus, dtype, stream: as for ss_scan_fwd.
 * out must not overlap state or the inputs.
 */
ss_status ss_state_update(float* state, const void* u, const void* delta, const float* A,
                          const void* B, const void* C, const float* D, const void* z,
                          const float* delta_bias, int delta_softplus, void* out,
                          int64_t batch, int64_t d_inner, int64_t d_state, ss_dtype dtype,
                          void* stream);

/* Decode with options: flags are SS_FLAG_* bits (0 = the ss_state_update operation). */
ss_status ss_state_update_ex(float* state, const void* u, const void* delta, const float* A,
                             const void* B, const void* C, const float* D, const void* z,
                             const float* delta_bias, int delta_softplus, void* out,
                             int64_t batch, int64_t d_inner, int64_t d_state, ss_dtype dtype,
                             uint32_t flags, void* stream);

/*
 * Backward of the prefill (first-order or exact-hold input term): given dout = dL/d out (and optionally
 * dh_last = dL/d h_last), the gradients of every input.  Reverse-mode differentiation of the
 * recurrence above (reading guide, "Método"), with the states recomputed from stored chunk-end
 * states rather than kept (reading guide, "Expansão de Estado Ciente de Hardware": recomputation
 * in the backward pass):
 *     lam_t[n] = gy_t C_t[n] + exp(dt_{t+1} A[d,n]) lam_{t+1}[n],  gy_t = dout_t silu(z_t)
 *     du_t = gy_t D + dt_t sum_n lam_t B_t,  ddt_t = sum_n lam_t (A e_t h_{t-1} + B_t u_t)
 *     ddelta_t = ddt_t sigmoid(delta_t + bias) (softplus') or ddt_t,  dz_t = dout_t y_t silu'(z_t)
 *     dB_t += lam_t dt_t u_t,  dC_t += gy_t h_t (over channels),  dA += lam_t dt_t e_t h_{t-1},
 *     dD += gy_t u_t,  ddelta_bias += ddelta_t,  dh0 = e_0 lam_0.
 *
 *   inputs            : exactly as given to ss_scan_fwd (u, delta, A, B, C, D, z, delta_bias,
 *                       delta_softplus, h0, sizes, dtype).
 *   dout              : (batch, seqlen, d_inner) io dtype, required.
 *   dh_last           : (batch, d_inner, d_state) float32; NULL means 0.
 *   du, ddelta        : (batch, seqlen, d_inner) io dtype, required, overwritten.
 *   dz                : (batch, seqlen, d_inner) io dtype, required iff z is given.
 *   dA                : (d_inner, d_state) float32, required, overwritten.
 *   dB, dC            : (batch, seqlen, d_state) float32, required, overwritten.
 *   dD, ddelta_bias   : (d_inner) float32, overwritten when non-NULL (the gradient at the given
 *                       D / bias, also when D or delta_bias is NULL, i.e. 0).
 *   dh0               : (batch, d_inner, d_state) float32, written when non-NULL.
 *   workspace         : 16-byte aligned device scratch of ss_scan_bwd_workspace_bytes() bytes,
 *                       required when that is non-zero (SS_ERR_INVALID_ARG if smaller): first
 *                       the chunk-end states, (batch, ceil(seqlen / 16), d_inner, d_state)
 *                       floats, then the partial sums of dB and dC per 16-channel block and of
 *                       dA, dD, ddelta_bias per batch row.  Without SS_FLAG_STATES_GIVEN the
 *                       call first writes the states there with a forward pass (a launch of its
 *                       own on the stream), then runs the reverse pass and two reductions.
 * dA, dB, dC, dD and ddelta_bias are sums over channels or batch rows: each workgroup writes its
 * partial sum and a second kernel adds the partials in a fixed order, so every output is
 * bit-for-bit reproducible.  flags: SS_FLAG_ZOH_EXACT gives the gradients of the exact-hold
 * input term g_t B_t u_t, g_t = (exp(dt_t A) - 1) / A (then ddt_t = sum_n lam_t e_t (A h_{t-1} +
 * B_t u_t), du_t = gy_t D + sum_n lam_t g_t B_t, dB_t += lam_t g_t u_t and dA adds
 * lam_t (dt e_t - g_t) / A B_t u_t); SS_FLAG_STATES_GIVEN as below, not together with the exact
 * hold (ss_scan_fwd_states saves first-order states): SS_ERR_UNSUPPORTED.  d_state above 64 ->
 * SS_ERR_UNSUPPORTED.
 * Outputs must not overlap inputs, each other or the workspace.
 */
ss_status ss_scan_bwd(const void* u, const void* delta, const float* A, const void* B,
                      const void* C, const float* D, const void* z, const float* delta_bias,
                      int delta_softplus, const float* h0, const void* dout,
                      const float* dh_last, void* du, void* ddelta, void* dz, float* dA,
                      float* dB, float* dC, float* dD, float* ddelta_bias, float* dh0,
                      int64_t batch, int64_t seqlen, int64_t d_inner, int64_t d_state,
                      ss_dtype dtype, void* workspace, size_t workspace_bytes, uint32_t flags,
                      void* stream);

/* Workspace bytes ss_scan_bwd needs for this shape (0 for an empty problem or d_state > 64).
 * With flags SS_FLAG_STATES_GIVEN the states part of the workspace is read, not written: it
 * must hold the states ss_scan_fwd_states wrote for the same u, delta, A, B, delta_bias,
 * delta_softplus, h0, sizes and dtype (C, D and z do not enter the states). */
size_t ss_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                   int64_t d_state, ss_dtype dtype);

/*
 * Multi-head scan with a scalar transition per head (the Mamba-2 form: IBM explainer, the
 * Mamba-2 block split into heads like multi-head attention, with B and C shared by groups of
 * heads as in grouped-query attention; Cartesia Mamba-3 post, the diagonal transition reduced to
 * a scalar times the identity).  For batch b, head h in group g = h / (nheads / ngroups), state n
 * and head channel p:
 *
 *     dt_t      = softplus(dt[b,t,h] + dt_bias[h])          (or the raw sum, softplus off)
 *     S_t[n,p]  = exp(dt_t * A[h]) * S_{t-1}[n,p] + dt_t * B[b,t,g,n] * x[b,t,h,p]
 *     y_t[p]    = sum_n C[b,t,g,n] * S_t[n,p] + D[h] * x[b,t,h,p]
 *     out       = y_t[p] * silu(z[b,t,h,p])                (when z is given)
 *
 *   x, z, out : (batch, seqlen, nheads, headdim), io dtype; z == NULL: no gate.
 *   dt        : (batch, seqlen, nheads), io dtype.
 *   B, C      : (batch, seqlen, ngroups, d_state), io dtype.
 *   A         : (nheads) float32, one transition per head.  D, dt_bias: (nheads) float32, NULL 0.
 *   h0, h_last: (batch, nheads, d_state, headdim) float32; NULL: zeros / not written.
 * nheads must be a multiple of ngroups (SS_ERR_INVALID_ARG); d_state outside 1..256 ->
 * SS_ERR_UNSUPPORTED.  Empty sizes are a no-op (h_last <- h0 or zeros).  out and h_last must not
 * overlap the inputs or each other.
 */
ss_status ss_scan2_fwd(const void* x, const void* dt, const float* A, const void* B,
                       const void* C, const float* D, const void* z, const float* dt_bias,
                       int dt_softplus, const float* h0, float* h_last, void* out,
                       int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                       int64_t ngroups, int64_t d_state, ss_dtype dtype, void* stream);

/*
 * Decode with the block's front end fused in (the one-token form of ss_scan_fwd_conv): takes
 * the block's x for this token and forms u = silu(conv_bias + sum_j conv_weight[d,j] *
 * window[j]) over the window [conv_state (the conv_k - 1 previous inputs, oldest first), x];
 * conv_state is then shifted in place (oldest dropped, x appended).
 *   conv_state   : (batch, conv_k - 1, d_inner) io dtype, read and overwritten IN PLACE
 *                  (required when conv_k > 1).
 *   x            : (batch, d_inner) io dtype.
 *   conv_weight, conv_bias, conv_k : as for ss_scan_fwd_conv.
 *   the rest     : as for ss_state_update_ex.
 * Needs d_state a multiple of 4 in 12..64 with 16-byte aligned state and A
 * (SS_ERR_UNSUPPORTED otherwise).  conv_state must not overlap state, out or the inputs.
 */
ss_status ss_state_update_conv(float* state, void* conv_state, const void* x,
                               const float* conv_weight, const float* conv_bias, int32_t conv_k,
                               const void* delta, const float* A, const void* B, const void* C,
                               const float* D, const void* z, const float* delta_bias,
                               int delta_softplus, void* out, int64_t batch, int64_t d_inner,
                               int64_t d_state, ss_dtype dtype, uint32_t flags, void* stream);

/* ---------------------------------------------------------------------------------------------
 * The recurrent block around a per-channel recurrence: a gated linear recurrence (one real state
 * per channel, its decay and its input both gated by the token), the layer norm with the residual
 * add in front of a block, and the causal depthwise convolution as an operator of its own, with
 * the gradients of all three and their one-token forms.  A block is
 *
 *     norm -> projection -> convolution -> gate projections -> recurrence -> projection
 *
 * where the projections are the caller's matrix products.  The convolution is separate here (and
 * not fused into the scan, as in ss_scan_fwd_conv) because the gates are projections of its
 * output.  Two arguments are shared:
 *   starts : (batch, seqlen) bytes or NULL.  A nonzero byte at step t begins a new sequence in
 *            the row: nothing before t reaches t or any later step, not even an infinity or a
 *            NaN, and no gradient flows back across it.  Rows that pack several sequences are
 *            the usual case.  A nonzero byte at t = 0 cuts off h0 / x_prev.
 *   io dtype : SS_F32 or SS_BF16 as above; parameters, states, statistics and every gradient
 *            that is a sum over tokens are float32, and all arithmetic is float32.
 * ------------------------------------------------------------------------------------------- */

/* Steps between two states that the forward saves for the backward. */
#define SS_GATED_CHUNK 64

/*
 * Gated linear recurrence.  For batch row b and channel d:
 *
 *     rg_t = sigmoid(r[b,t,d] + r_bias[d])       how far the state decays at this token
 *     ig_t = sigmoid(i[b,t,d] + i_bias[d])       how much of the token enters it
 *     a_t  = exp(A[d] * rg_t)                    A <= 0: a decay in (0, 1]
 *     h_t  = a_t h_{t-1} + sqrt(1 - a_t^2) ig_t x[b,t,d]       (no h_{t-1} where starts[b,t])
 *     out  = h_t * silu(z[b,t,d])                (when z is given)
 *
 *   x, r, i, z, out  : (batch, seqlen, d_inner) io dtype.  z == NULL: out = h.
 *   A                : (d_inner) float32, not above 0 (a channel with A > 0 gives NaN).
 *   r_bias, i_bias   : (d_inner) float32, NULL means 0.
 *   h0, h_last       : (batch, d_inner) float32; NULL: zeros / not written.
 *   states           : NULL, or (batch, ceil(seqlen / SS_GATED_CHUNK), d_inner) float32: the
 *                      state after every SS_GATED_CHUNK steps (and after the last step), for
 *                      ss_gated_scan_bwd.  ss_gated_scan_states_bytes() bytes.
 *   workspace        : ss_gated_scan_fwd_workspace_bytes() bytes, 16-byte aligned; may be NULL
 *                      when that is 0.  Its contents need no preparation and mean nothing after
 *                      the call; calls that may run at the same time need one each.
 * 1 - a^2 is formed without cancellation (as -expm1(2 A rg)).  Results do not depend on timing or
 * on the order in which workgroups run: two runs agree bit for bit.  They do depend, by rounding,
 * on where a step lies in its row: a sequence behind a start and the same one in a call of its own
 * agree to a few float32 roundings per step.  A decay below 2^-126 counts as 0 and a product of
 * decays below it as 2^-126: an error of at most 2^-126 times the state before.
 * Outputs must not overlap the inputs, each other or the workspace (SS_ERR_INVALID_ARG); d_inner
 * above 2^24 or seqlen above 2^31 - 1 -> SS_ERR_UNSUPPORTED.  Empty sizes are a no-op (with
 * seqlen == 0, h_last receives h0, or zeros).
 */
ss_status ss_gated_scan_fwd(const void* x, const void* r, const void* i, const float* A,
                            const float* r_bias, const float* i_bias, const void* z,
                            const uint8_t* starts, const float* h0, float* h_last, void* out,
                            float* states, int64_t batch, int64_t seqlen, int64_t d_inner,
                            ss_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream);
size_t ss_gated_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                         ss_dtype dtype);
size_t ss_gated_scan_states_bytes(int64_t batch, int64_t seqlen, int64_t d_inner);

/*
 * Gradients of ss_gated_scan_fwd for the upstream gradients dout (io dtype, required) and
 * dh_last (float32, NULL: 0), by the adjoint recurrence
 *
 *     lam_t = dout_t silu(z_t) + a_{t+1} lam_{t+1}       (no second term where starts[b,t+1])
 *     dx = lam s ig;   di = lam s x ig (1 - ig);   dz = dout h silu'(z);   s = sqrt(1 - a^2)
 *     dr = dl A rg (1 - rg);   dA = sum dl rg;   dl = lam (a h_{t-1} - ig x a^2 / s)
 *     dr_bias = sum dr;   di_bias = sum di;   dh0 = a_0 lam_0 (0 where starts[b,0])
 * Where a = 1 exactly (s = 0) the second term of dl counts as 0: a gate that has underflowed
 * passes no gradient.
 *   states            : what ss_gated_scan_fwd saved for the same inputs, or NULL: the states
 *                       are then recomputed by a pass of its own (into the workspace).
 *   dx, dr, di        : (batch, seqlen, d_inner) io dtype, required; dz likewise with z (without
 *                       z it is not written).
 *   dA                : (d_inner) float32, required.  dr_bias, di_bias: (d_inner) float32, NULL:
 *                       not written.  Sums over batch rows and steps, in a fixed order: two runs
 *                       agree bit for bit.  Zeros when there are no tokens.
 *   dh0               : (batch, d_inner) float32, NULL: not written.
 *   workspace         : ss_gated_scan_bwd_workspace_bytes(..., states != NULL) bytes, 16-byte
 *                       aligned; the same rules as the forward's.
 */
ss_status ss_gated_scan_bwd(const void* x, const void* r, const void* i, const float* A,
                            const float* r_bias, const float* i_bias, const void* z,
                            const uint8_t* starts, const float* h0, const void* dout,
                            const float* dh_last, const float* states, void* dx, void* dr,
                            void* di, void* dz, float* dA, float* dr_bias, float* di_bias,
                            float* dh0, int64_t batch, int64_t seqlen, int64_t d_inner,
                            ss_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream);
size_t ss_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                         ss_dtype dtype, int states_given);

/*
 * One token of the gated linear recurrence: state (batch, d_inner) float32 is advanced IN PLACE;
 * x, r, i, z, out: (batch, d_inner) io dtype; the rest as in ss_gated_scan_fwd.  state and out
 * must not overlap the inputs or each other.
 */
ss_status ss_gated_state_update(float* state, const void* x, const void* r, const void* i,
                                const float* A, const float* r_bias, const float* i_bias,
                                const void* z, void* out, int64_t batch, int64_t d_inner,
                                ss_dtype dtype, void* stream);

/*
 * Layer norm over the last axis, with the residual add in front of it:
 *
 *     s = x + residual;   mu = mean(s);   rstd = 1 / sqrt(mean((s - mu)^2) + eps)
 *     out = (s - mu) rstd weight + bias
 *
 *   x, out           : (rows, dim) io dtype.
 *   residual, sum    : (rows, dim) float32.  The residual stream is float32 whatever the io
 *                      dtype: it collects one term per layer, and rounding each partial sum to
 *                      bfloat16 would lose what the deep layers add.  residual == NULL: s = x.
 *                      sum == NULL: s is not written.  (residual NULL with sum given widens x.)
 *   weight, bias     : (dim) float32, NULL means 1 / 0.
 *   mean, rstd       : (rows) float32 statistics for the backward; NULL: not written.
 *   eps              : not negative (SS_ERR_INVALID_ARG).
 * The variance is the mean of squared differences from the mean, not a difference of moments.
 * Outputs must not overlap the inputs or each other.  rows == 0 or dim == 0 is a no-op.
 * dim above 2^24 -> SS_ERR_UNSUPPORTED.
 */
ss_status ss_layer_norm_fwd(const void* x, const float* residual, const float* weight,
                            const float* bias, float eps, void* out, float* sum, float* mean,
                            float* rstd, int64_t rows, int64_t dim, ss_dtype dtype,
                            void* stream);

/*
 * Gradients of ss_layer_norm_fwd: with xh = (s - mean) rstd and g = dout weight,
 *
 *     ds      = rstd (g - mean(g) - xh mean(g xh)) + dsum
 *     dweight = sum over rows of dout xh;   dbias = sum over rows of dout
 *
 *   dout       : (rows, dim) in `dtype`.
 *   s          : (rows, dim) in `s_dtype`: x itself (s_dtype == dtype) or the float32 sum the
 *                forward wrote.
 *   mean, rstd : as the forward wrote them.      weight: as the forward's.
 *   dsum       : (rows, dim) float32 upstream gradient of sum, NULL: 0.
 *   dx         : ds in `dtype`, the gradient of x.  dresidual: ds in float32, the gradient of
 *                residual.  At least one is required.
 *   dweight, dbias : (dim) float32, NULL: not written.  Summed in a fixed order: two runs agree
 *                bit for bit.  Zeros when rows == 0.
 *   workspace  : ss_layer_norm_bwd_workspace_bytes() bytes, 16-byte aligned; one per call that
 *                may run at the same time.
 */
ss_status ss_layer_norm_bwd(const void* dout, const void* s, ss_dtype s_dtype,
                            const float* weight, const float* mean, const float* rstd,
                            const float* dsum, void* dx, float* dresidual, float* dweight,
                            float* dbias, int64_t rows, int64_t dim, ss_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream);
size_t ss_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim);

/*
 * Causal depthwise convolution, the front end of ss_scan_fwd_conv as an operator of its own:
 *
 *     p[b,t,d] = bias[d] + sum_{j<k} weight[d,j] x[b, t-(k-1)+j, d];   out = silu(p) or p
 *
 *   x, out       : (batch, seqlen, d_inner) io dtype.
 *   weight       : (d_inner, k) float32, k in 1..4 (SS_ERR_UNSUPPORTED otherwise).
 *   bias         : (d_inner) float32, NULL means 0.
 *   x_prev       : (batch, k-1, d_inner) io dtype, the inputs before t = 0 (oldest first), NULL:
 *                  zeros.
 *   silu         : nonzero -> out = silu(p), zero -> out = p.
 * out must not overlap the inputs.  d_inner above 2^24 or seqlen above 2^31 - 1 ->
 * SS_ERR_UNSUPPORTED.  Empty sizes are a no-op.
 */
ss_status ss_causal_conv_fwd(const void* x, const float* weight, const float* bias,
                             const void* x_prev, const uint8_t* starts, int silu, void* out,
                             int64_t batch, int64_t seqlen, int64_t d_inner, int32_t k,
                             ss_dtype dtype, void* stream);

/*
 * Gradients of ss_causal_conv_fwd, with g = dout silu'(p) (p recomputed) or dout:
 *
 *     dx_t = sum_j weight[j] g_{t+(k-1)-j};   dweight[j] = sum g_t x_{t-(k-1)+j};
 *     dbias = sum g;   dx_prev as dx at the steps before t = 0    (none across a start)
 *
 *   dx             : (batch, seqlen, d_inner) io dtype, required.
 *   dweight        : (d_inner, k) float32, required.  dbias: (d_inner) float32, NULL: not
 *                    written.  Summed over batch rows and steps in a fixed order: two runs agree
 *                    bit for bit.  Zeros when there are no tokens.
 *   dx_prev        : (batch, k-1, d_inner) io dtype, NULL: not written (needs x_prev).
 *   workspace      : ss_causal_conv_bwd_workspace_bytes() bytes, 16-byte aligned; one per call
 *                    that may run at the same time.
 */
ss_status ss_causal_conv_bwd(const void* x, const float* weight, const float* bias,
                             const void* x_prev, const uint8_t* starts, int silu,
                             const void* dout, void* dx, float* dweight, float* dbias,
                             void* dx_prev, int64_t batch, int64_t seqlen, int64_t d_inner,
                             int32_t k, ss_dtype dtype, void* workspace, size_t workspace_bytes,
                             void* stream);
size_t ss_causal_conv_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                          int32_t k, ss_dtype dtype);

/*
 * One token of the convolution: the window is [conv_state (batch, k-1, d_inner), x (batch,
 * d_inner)]; conv_state is shifted IN PLACE (oldest dropped, x appended).  conv_state may be
 * NULL when k == 1; conv_state and out must not overlap the inputs or each other.
 */
ss_status ss_causal_conv_update(void* conv_state, const void* x, const float* weight,
                                const float* bias, int silu, void* out, int64_t batch,
                                int64_t d_inner, int32_t k, ss_dtype dtype, void* stream);

/* ---------------------------------------------------------------------------------------------
 * The block around the multi-head scan (ss_scan2_fwd): the scan's next token with the convolution
 * in front of it, its gradients, the RMS norm in front of a block (which adds the block before to
 * the residual stream), the gated RMS norm behind the scan, and dropout.  A block is
 *
 *     norm -> projection [z | x B C | dt] -> convolution -> scan -> gated norm -> projection
 *
 * where the projections are the caller's matrix products.  io dtype as above; parameters, states,
 * statistics and every gradient that is a sum over tokens are float32, and so is all arithmetic.
 * Some inputs are parts of a projection's rows: those have a `_stride`, the elements from one row
 * to the next (at least the row's own; other arrays are contiguous).
 * ------------------------------------------------------------------------------------------- */

/*
 * Gradients of ss_scan2_fwd for the upstream gradients dout (io dtype, required) and dh_last
 * (float32, NULL: 0), with lam_t = dL/dS_t:
 *
 *     gy_t  = dout_t silu(z_t);    lam_t = C_t gy_t^T + a_{t+1} lam_{t+1};   a_t = exp(dt_t A)
 *     dx_t  = D gy_t + dt_t lam_t^T B_t;           dz_t = dout_t y_t silu'(z_t)
 *     dB_t  = sum over the group's heads of dt_t lam_t x_t;   dC_t = sum of S_t gy_t
 *     dl_t  = <lam_t, a_t S_{t-1}>;   ddt_t = (A dl_t + x_t . lam_t^T B_t) softplus'(dt_t + bias)
 *     dA = sum dt_t dl_t;   dD = sum gy_t . x_t;   ddt_bias = sum ddt_t;   dh0 = a_0 lam_0
 *
 *   x .. h0, sizes    : exactly as given to ss_scan2_fwd.
 *   dx, ddt, dB, dC   : in the io dtype and the shapes of x, dt, B and C, required; dz likewise
 *                       with z (without z it is not written).  dB and dC are added over the heads
 *                       in float32 and rounded once: they go on as rows of the convolution's or
 *                       the projection's upstream gradient.
 *   dA                : (nheads) float32, required.  dD, ddt_bias: (nheads) float32, NULL: not
 *                       written (the gradient at the given D / bias, also when those are NULL,
 *                       i.e. 0).  Sums in a fixed order: two runs agree bit for bit.  Zeros when
 *                       there are no tokens.
 *   dh0               : (batch, nheads, d_state, headdim) float32, NULL: not written.
 *   workspace         : ss_scan2_bwd_workspace_bytes() bytes, 16-byte aligned: first the states
 *                       before and the adjoints behind every 64 steps.  Its contents need no
 *                       preparation and mean nothing after the call; calls that may run at the
 *                       same time need one each.
 * nheads == 0 is a no-op (dB and dC are not written).  d_state outside 1..256, headdim or nheads
 * above 2^24 or seqlen above 2^31 - 1 -> SS_ERR_UNSUPPORTED.  Outputs must not overlap inputs, each
 * other or the workspace.
 * dA, dD, ddt_bias and dh0 are what float32 products and sums give, for either io dtype.  With bf16
 * io, headdim 64 and 64 or 128 states the products run on bf16 parts: three of a float32 operand (all
 * of it) towards those, two (2^-17 of it) towards gradients that are rounded to bf16.
 * The products are formed for 64 steps at a time, pairs in the wrong order times 0: an infinity or
 * a NaN at a step reaches the gradients of other steps of its 64, also ones that do not depend on
 * it (as in ss_scan2_fwd's matrix form).
 */
ss_status ss_scan2_bwd(const void* x, const void* dt, const float* A, const void* B,
                       const void* C, const float* D, const void* z, const float* dt_bias,
                       int dt_softplus, const float* h0, const void* dout, const float* dh_last,
                       void* dx, void* ddt, void* dz, float* dA, void* dB, void* dC, float* dD,
                       float* ddt_bias, float* dh0, int64_t batch, int64_t seqlen,
                       int64_t nheads, int64_t headdim, int64_t ngroups, int64_t d_state,
                       ss_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);
size_t ss_scan2_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads,
                                    int64_t headdim, int64_t ngroups, int64_t d_state,
                                    ss_dtype dtype);

/*
 * One token of ss_scan2_fwd: state (batch, nheads, d_state, headdim) float32 (the layout of
 * h_last) is advanced IN PLACE; x, z, out: (batch, nheads, headdim), dt: (batch, nheads), B, C:
 * (batch, ngroups, d_state), io dtype; the rest as in ss_scan2_fwd.  state and out must not
 * overlap the inputs or each other.
 */
ss_status ss_scan2_state_update(float* state, const void* x, const void* dt, const float* A,
                                const void* B, const void* C, const float* D, const void* z,
                                const float* dt_bias, int dt_softplus, void* out, int64_t batch,
                                int64_t nheads, int64_t headdim, int64_t ngroups,
                                int64_t d_state, ss_dtype dtype, void* stream);

/*
 * The same with the convolution in front: x, B and C are what ss_causal_conv_update (with silu)
 * makes of xbc, whose rows hold [x (nheads headdim) | B (ngroups d_state) | C (ngroups d_state)],
 * `width` columns together; between the convolution and the scan they stay float32.
 *   xbc        : (batch, width) io dtype, rows xbc_stride elements apart.
 *   conv_state : (batch, conv_k - 1, width) io dtype, the window before this token (oldest
 *                first), shifted IN PLACE.  May be NULL when conv_k == 1.
 *   conv_weight: (width, conv_k) float32, conv_k in 1..4 (SS_ERR_UNSUPPORTED otherwise);
 *                conv_bias: (width) float32, NULL means 0.
 *   dt, z      : (batch, nheads) and (batch, nheads headdim), rows dt_stride and z_stride
 *                elements apart (z_stride means nothing without z).
 *   workspace  : ss_scan2_state_update_conv_workspace_bytes() bytes, 16-byte aligned; one per
 *                call that may run at the same time.
 * batch, nheads or headdim == 0 is a no-op (the window is not shifted either).
 * state, conv_state and out must not overlap the inputs, each other or the workspace.
 */
ss_status ss_scan2_state_update_conv(float* state, void* conv_state, const void* xbc,
                                     int64_t xbc_stride, const float* conv_weight,
                                     const float* conv_bias, int32_t conv_k, const void* dt,
                                     int64_t dt_stride, const float* A, const float* D,
                                     const void* z, int64_t z_stride, const float* dt_bias,
                                     int dt_softplus, void* out, int64_t batch, int64_t nheads,
                                     int64_t headdim, int64_t ngroups, int64_t d_state,
                                     ss_dtype dtype, void* workspace, size_t workspace_bytes,
                                     void* stream);
size_t ss_scan2_state_update_conv_workspace_bytes(int64_t batch, int64_t nheads, int64_t headdim,
                                                  int64_t ngroups, int64_t d_state);

/*
 * RMS norm over the last axis, with a block's output added to the residual stream before it:
 *
 *     b = x, or x / sqrt(mean(x^2) + eps)  (norm_branch: the norm behind the block)
 *     s = residual + drop(scale b);   rstd = 1 / sqrt(mean(s^2) + eps);   out = s rstd weight
 *
 *   x, out           : (rows, dim) io dtype.
 *   residual, sum    : (rows, dim) float32 (as in ss_layer_norm_fwd).  residual NULL: 0.  sum
 *                      NULL: s is not written.
 *   weight, scale    : (dim) float32, NULL means 1.  `scale` is the block's learned residual scale
 *                      or, with norm_branch, that norm's weight.
 *   p, rng           : dropout as in ss_dropout; p == 0: none (rng is not read and may be NULL).
 *   rstd, branch_rstd: (rows) float32 statistics for the backward; NULL: not written (branch_rstd
 *                      not without norm_branch either).
 *   eps              : not negative (SS_ERR_INVALID_ARG).
 * Outputs must not overlap the inputs or each other.  rows == 0 or dim == 0 is a no-op.
 * dim above 2^24 -> SS_ERR_UNSUPPORTED; rows above 2^31 - 1 -> SS_ERR_INVALID_ARG.
 */
ss_status ss_rms_norm_fwd(const void* x, const float* residual, const float* weight,
                          const float* scale, int norm_branch, double p, const uint64_t* rng,
                          float eps, void* out, float* sum, float* rstd, float* branch_rstd,
                          int64_t rows, int64_t dim, ss_dtype dtype, void* stream);

/*
 * Gradients of ss_rms_norm_fwd, with sh = s rstd, g = dout weight and b as there:
 *
 *     ds = rstd (g - sh mean(g sh)) + dsum;   db = drop(ds);   dweight = sum of dout sh
 *     dscale = sum of db b;   dx = db scale, or through the norm: branch_rstd (db scale -
 *     b mean(db scale b))
 *
 *   s            : (rows, dim) in `s_dtype`: x itself (s_dtype == dtype, where the forward had
 *                  none of residual, scale, norm_branch and dropout) or the float32 sum it wrote
 *                  (SS_ERR_INVALID_ARG otherwise, where the call shows it).
 *   x            : as the forward's; read for dscale and with norm_branch, else it may be NULL.
 *   rstd, branch_rstd : as the forward wrote them (branch_rstd with norm_branch only).
 *   weight, scale, p, rng : as the forward's.
 *   dsum         : (rows, dim) float32 upstream gradient of sum, NULL: 0.
 *   dx, dresidual: the gradients of x (in `dtype`) and of residual (ds, float32).  At least one is
 *                  required.
 *   dweight, dscale : (dim) float32, NULL: not written.  Summed in a fixed order: two runs agree
 *                  bit for bit.  Zeros when rows == 0.
 *   workspace    : ss_rms_norm_bwd_workspace_bytes() bytes, 16-byte aligned, with dweight or
 *                  dscale; one per call that may run at the same time.
 */
ss_status ss_rms_norm_bwd(const void* dout, const void* s, ss_dtype s_dtype,
                          const float* weight, const float* rstd, const void* x,
                          const float* scale, int norm_branch, const float* branch_rstd,
                          double p, const uint64_t* rng, const float* dsum, void* dx,
                          float* dresidual, float* dweight, float* dscale, int64_t rows,
                          int64_t dim, ss_dtype dtype, void* workspace, size_t workspace_bytes,
                          void* stream);
size_t ss_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t dim);

/*
 * RMS norm with the output gate, over each of `groups` runs of dim / groups columns of a row:
 *
 *     gate_first: u = x silu(z);  out = u rstd weight       else: u = x;  out = u rstd weight silu(z)
 *     rstd = 1 / sqrt(mean over the run of u^2 + eps)
 *
 *   x, out   : (rows, dim) io dtype.      z : the same, rows z_stride elements apart; NULL: no gate.
 *   weight   : (dim) float32, NULL means 1.
 *   rstd     : (rows, groups) float32 statistics for the backward; NULL: not written.
 * dim not a multiple of groups, or rows * groups above 2^31 - 1 or groups above 2^20 ->
 * SS_ERR_INVALID_ARG; the rest as in ss_rms_norm_fwd.
 */
ss_status ss_gated_norm_fwd(const void* x, const void* z, int64_t z_stride, const float* weight,
                            int gate_first, float eps, void* out, float* rstd, int64_t rows,
                            int64_t dim, int64_t groups, ss_dtype dtype, void* stream);

/*
 * Gradients of ss_gated_norm_fwd.  dx: (rows, dim) io dtype, required; dz likewise with z
 * (contiguous; without z it is not written); dweight: (dim) float32, NULL: not written, summed in a
 * fixed order, zeros when rows == 0.  rstd as the forward wrote it.  workspace:
 * ss_gated_norm_bwd_workspace_bytes() bytes, 16-byte aligned, with dweight; one per call that may
 * run at the same time.
 */
ss_status ss_gated_norm_bwd(const void* dout, const void* x, const void* z, int64_t z_stride,
                            const float* weight, const float* rstd, int gate_first, void* dx,
                            void* dz, float* dweight, int64_t rows, int64_t dim, int64_t groups,
                            ss_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream);
size_t ss_gated_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t groups);

/*
 * Dropout: out = x / (1 - q) where the element is kept, 0 (exactly, whatever x is) where it is
 * dropped.  q is p rounded to a multiple of 2^-16, p in 0..1 (SS_ERR_INVALID_ARG otherwise).
 *   x, out : (rows, dim) io dtype.
 *   rng    : two 64-bit numbers in DEVICE memory, a seed and an offset, read by the kernel (a
 *            captured call draws anew when the caller has advanced them).  Required.
 * The mask is not stored: it is a function of rng and of the element's row and column alone
 * (Philox4x32-10 under the key `seed`: 16 bits per element, eight columns a counter (column / 8,
 * row, offset)), the same in ss_dropout, ss_rms_norm_fwd and ss_rms_norm_bwd.  The gradient is this
 * call on the upstream gradient.  Draws that are to be independent need another offset or seed.
 * out must not overlap x.  rows == 0 or dim == 0 is a no-op; limits as in ss_rms_norm_fwd.
 */
ss_status ss_dropout(const void* x, void* out, double p, const uint64_t* rng, int64_t rows,
                     int64_t dim, ss_dtype dtype, void* stream);

/* Static description of a status code. */
const char* ss_status_string(ss_status s);

/* Thread-local detail of the last non-OK status returned on this thread ("" if none). */
const char* ss_last_error(void);

/* Library ABI version (major * 100 + minor). */
int ss_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SS_SCAN_H */
