// ss_block_api.hip -- the C ABI of the recurrent block's operators (declared in
// include/ss_scan.h): argument checking, workspace sizes and dispatch.  No allocation, no
// synchronisation, no printing, nothing that throws.
#include <math.h>

#include "ss_block.h"
#include "ss_host.h"

namespace {

using namespace ss::host;

constexpr int64_t kMaxWidth = int64_t(1) << 24;
constexpr int64_t kMaxSteps = 0x7fffffff;
constexpr int64_t kMaxGrid = 0x7fffffff;

// One array argument: its extent, and whether it may be NULL.
struct Arr {
  const char* name;
  const void* p;
  int64_t elems, esize;
  bool required;
};

// Presence and alignment of every array, then no output over an input or another output.
ss_status check_arrays(const Arr* in, int n_in, const Arr* out, int n_out) {
  for (int k = 0; k < n_in + n_out; ++k) {
    const Arr& a = k < n_in ? in[k] : out[k - n_in];
    if (a.required && !a.p) return fail(SS_ERR_INVALID_ARG, "%s is NULL", a.name);
    if (a.p && !aligned(a.p, a.esize))
      return fail(SS_ERR_UNSUPPORTED, "%s pointer %p not aligned to its %lld-byte element",
                  a.name, a.p, static_cast<long long>(a.esize));
  }
  for (int k = 0; k < n_out; ++k) {
    const Range o = range(out[k].name, out[k].p, out[k].elems, out[k].esize);
    for (int j = 0; j < n_in; ++j)
      if (overlap(o, range(in[j].name, in[j].p, in[j].elems, in[j].esize)))
        return fail(SS_ERR_INVALID_ARG, "%s overlaps %s", out[k].name, in[j].name);
    for (int j = k + 1; j < n_out; ++j)
      if (overlap(o, range(out[j].name, out[j].p, out[j].elems, out[j].esize)))
        return fail(SS_ERR_INVALID_ARG, "%s overlaps %s", out[k].name, out[j].name);
  }
  return SS_OK;
}

// Sizes of a (batch, seqlen, d_inner) operator: `elems` fits 64-bit byte offsets.
ss_status check_sizes(int64_t batch, int64_t seqlen, int64_t d_inner, int64_t* elems) {
  if (batch < 0 || seqlen < 0 || d_inner < 0)
    return fail(SS_ERR_INVALID_ARG, "negative size (batch=%lld seqlen=%lld d_inner=%lld)",
                static_cast<long long>(batch), static_cast<long long>(seqlen),
                static_cast<long long>(d_inner));
  if (d_inner > kMaxWidth)
    return fail(SS_ERR_UNSUPPORTED, "d_inner=%lld above 16777216",
                static_cast<long long>(d_inner));
  if (seqlen > kMaxSteps)
    return fail(SS_ERR_UNSUPPORTED, "seqlen=%lld above 2147483647",
                static_cast<long long>(seqlen));
  int64_t n, m;
  // (seqlen + 8) covers the window before the sequence and the partial sums of a chunk
  if (!mul_ok(batch, d_inner, &n) || !mul_ok(n, seqlen + 8, &n) || !mul_ok(n, 64, &m))
    return fail(SS_ERR_INVALID_ARG, "sizes overflow 64-bit byte offsets");
  if ((n + 63) / 64 > kMaxGrid)
    return fail(SS_ERR_INVALID_ARG, "too many elements (batch * seqlen * d_inner)");
  *elems = batch * seqlen * d_inner;
  return SS_OK;
}

ss_status check_workspace(const void* ws, size_t have, size_t need, const char* query) {
  if (need == 0) return SS_OK;
  if (!ws || have < need)
    return fail(SS_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu bytes needed "
                "(%s)", ws ? have : size_t(0), need, query);
  if (!aligned(ws, 16))
    return fail(SS_ERR_UNSUPPORTED, "workspace pointer %p not 16-byte aligned", ws);
  return SS_OK;
}

ss_status launched(hipError_t e) {
  return e == hipSuccess ? ok() : fail(SS_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

bool sizes_ok(int64_t batch, int64_t seqlen, int64_t d_inner) {
  int64_t n;
  return batch > 0 && seqlen > 0 && d_inner > 0 && d_inner <= kMaxWidth && seqlen <= kMaxSteps &&
         mul_ok(batch, d_inner, &n) && mul_ok(n, seqlen + 8, &n) && n / 64 < kMaxGrid;
}

// A launch counts its threads in 32 bits.
ss_status check_grid(int64_t blocks, int64_t threads) {
  if (blocks > 0xffffffffll / threads)
    return fail(SS_ERR_INVALID_ARG, "too many elements for one launch");
  return SS_OK;
}
// The recurrence: one workgroup per tile and 64 channels, one wave per `per_wave` steps in it.
ss_status check_tiles(int64_t batch, int64_t seqlen, int64_t d_inner, int64_t tile,
                      int64_t per_wave) {
  const int64_t waves = seqlen > tile ? tile / per_wave : (seqlen + per_wave - 1) / per_wave;
  return check_grid(batch * ((d_inner + 63) / 64) * ((seqlen + tile - 1) / tile),
                    64 * (waves > 0 ? waves : 1));
}

int64_t chunks_of(int64_t seqlen) { return (seqlen + SS_GATED_CHUNK - 1) / SS_GATED_CHUNK; }

}  // namespace

extern "C" {

// (The workspaces hold float32 sums and states only: their sizes do not depend on the io dtype that
// the queries take, as the scan's do.)
size_t ss_gated_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                         ss_dtype) {
  if (!sizes_ok(batch, seqlen, d_inner)) return 0;
  return ss::gated_fwd_ws_bytes(batch, seqlen, d_inner);
}

size_t ss_gated_scan_states_bytes(int64_t batch, int64_t seqlen, int64_t d_inner) {
  if (!sizes_ok(batch, seqlen, d_inner)) return 0;
  return static_cast<size_t>(batch * chunks_of(seqlen) * d_inner) * sizeof(float);
}

ss_status ss_gated_scan_fwd(const void* x, const void* r, const void* i, const float* A,
                            const float* r_bias, const float* i_bias, const void* z,
                            const uint8_t* starts, const float* h0, float* h_last, void* out,
                            float* states, int64_t batch, int64_t seqlen, int64_t d_inner,
                            ss_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = check_sizes(batch, seqlen, d_inner, &n)) != SS_OK) return s;
  const int64_t rows = batch * d_inner;
  if (rows == 0) return ok();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (seqlen == 0) {
    if (!h_last) return ok();
    const Arr in[] = {{"h0", h0, rows, 4, false}}, out1[] = {{"h_last", h_last, rows, 4, true}};
    if ((s = check_arrays(in, 1, out1, 1)) != SS_OK) return s;
    return launched(h0 ? ss::launch_copy(h_last, h0, rows, st) : ss::launch_zero(h_last, rows, st));
  }
  if ((s = check_tiles(batch, seqlen, d_inner, ss::kGatedFwdTile, ss::kGatedFwdSteps)) != SS_OK)
    return s;
  const size_t need = ss::gated_fwd_ws_bytes(batch, seqlen, d_inner);
  const Arr in[] = {{"x", x, n, es, true}, {"r", r, n, es, true}, {"i", i, n, es, true},
                    {"A", A, d_inner, 4, true}, {"r_bias", r_bias, d_inner, 4, false},
                    {"i_bias", i_bias, d_inner, 4, false}, {"z", z, n, es, false},
                    {"starts", starts, batch * seqlen, 1, false}, {"h0", h0, rows, 4, false}};
  const Arr outs[] = {{"out", out, n, es, true}, {"h_last", h_last, rows, 4, false},
                      {"states", states, batch * chunks_of(seqlen) * d_inner, 4, false},
                      {"workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1,
                       false}};
  if ((s = check_arrays(in, 9, outs, 4)) != SS_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "ss_gated_scan_fwd_workspace_bytes")) != SS_OK)
    return s;
  ss::GatedArgs a{};
  a.x = x; a.r = r; a.i = i; a.z = z; a.A = A; a.r_bias = r_bias; a.i_bias = i_bias;
  a.starts = starts; a.h0 = h0; a.h_last = h_last; a.out = out; a.states = states;
  a.workspace = workspace;
  a.batch = batch; a.seqlen = seqlen; a.d_inner = d_inner; a.n_chunks = chunks_of(seqlen);
  return launched(ss::launch_gated_fwd(a, dtype == SS_BF16, st));
}

size_t ss_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                         ss_dtype, int states_given) {
  if (!sizes_ok(batch, seqlen, d_inner)) return 0;
  return ss::gated_bwd_ws_bytes(batch, seqlen, d_inner, states_given != 0);
}

ss_status ss_gated_scan_bwd(const void* x, const void* r, const void* i, const float* A,
                            const float* r_bias, const float* i_bias, const void* z,
                            const uint8_t* starts, const float* h0, const void* dout,
                            const float* dh_last, const float* states, void* dx, void* dr,
                            void* di, void* dz, float* dA, float* dr_bias, float* di_bias,
                            float* dh0, int64_t batch, int64_t seqlen, int64_t d_inner,
                            ss_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = check_sizes(batch, seqlen, d_inner, &n)) != SS_OK) return s;
  if (d_inner == 0) return ok();
  if ((s = check_tiles(batch, seqlen, d_inner, SS_GATED_CHUNK, ss::kGatedBwdSteps)) != SS_OK)
    return s;
  const int64_t rows = batch * d_inner;
  const bool some = n > 0;
  const size_t need =
      some ? ss::gated_bwd_ws_bytes(batch, seqlen, d_inner, states != nullptr) : 0;
  const Arr in[] = {{"x", x, n, es, some}, {"r", r, n, es, some}, {"i", i, n, es, some},
                    {"A", A, d_inner, 4, true}, {"r_bias", r_bias, d_inner, 4, false},
                    {"i_bias", i_bias, d_inner, 4, false}, {"z", z, n, es, false},
                    {"starts", starts, batch * seqlen, 1, false}, {"h0", h0, rows, 4, false},
                    {"dout", dout, n, es, some}, {"dh_last", dh_last, rows, 4, false},
                    {"states", states, batch * chunks_of(seqlen) * d_inner, 4, false}};
  const Arr outs[] = {{"dx", dx, n, es, some}, {"dr", dr, n, es, some}, {"di", di, n, es, some},
                      {"dz", z ? dz : nullptr, n, es, some && z}, {"dA", dA, d_inner, 4, true},
                      {"dr_bias", dr_bias, d_inner, 4, false},
                      {"di_bias", di_bias, d_inner, 4, false}, {"dh0", dh0, rows, 4, false},
                      {"workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1,
                       false}};
  if ((s = check_arrays(in, 12, outs, 9)) != SS_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "ss_gated_scan_bwd_workspace_bytes")) != SS_OK)
    return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (!some) {
    hipError_t e = ss::launch_zero(dA, d_inner, st);
    if (e == hipSuccess && dr_bias) e = ss::launch_zero(dr_bias, d_inner, st);
    if (e == hipSuccess && di_bias) e = ss::launch_zero(di_bias, d_inner, st);
    if (e == hipSuccess && dh0 && rows)
      e = dh_last ? ss::launch_copy(dh0, dh_last, rows, st) : ss::launch_zero(dh0, rows, st);
    return launched(e);
  }
  ss::GatedArgs a{};
  a.x = x; a.r = r; a.i = i; a.z = z; a.A = A; a.r_bias = r_bias; a.i_bias = i_bias;
  a.starts = starts; a.h0 = h0; a.dout = dout; a.dh_last = dh_last;
  a.states = const_cast<float*>(states);
  a.dx = dx; a.dr = dr; a.di = di; a.dz = dz; a.dA = dA; a.dr_bias = dr_bias;
  a.di_bias = di_bias; a.dh0 = dh0; a.workspace = workspace;
  a.batch = batch; a.seqlen = seqlen; a.d_inner = d_inner; a.n_chunks = chunks_of(seqlen);
  return launched(ss::launch_gated_bwd(a, dtype == SS_BF16, st));
}

ss_status ss_gated_state_update(float* state, const void* x, const void* r, const void* i,
                                const float* A, const float* r_bias, const float* i_bias,
                                const void* z, void* out, int64_t batch, int64_t d_inner,
                                ss_dtype dtype, void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = check_sizes(batch, 1, d_inner, &n)) != SS_OK) return s;
  if (n == 0) return ok();
  if ((s = check_grid((n + 255) / 256, 256)) != SS_OK) return s;
  const Arr in[] = {{"x", x, n, es, true}, {"r", r, n, es, true}, {"i", i, n, es, true},
                    {"A", A, d_inner, 4, true}, {"r_bias", r_bias, d_inner, 4, false},
                    {"i_bias", i_bias, d_inner, 4, false}, {"z", z, n, es, false}};
  const Arr outs[] = {{"state", state, n, 4, true}, {"out", out, n, es, true}};
  if ((s = check_arrays(in, 7, outs, 2)) != SS_OK) return s;
  ss::GatedStepArgs a{};
  a.state = state; a.x = x; a.r = r; a.i = i; a.z = z; a.A = A; a.r_bias = r_bias;
  a.i_bias = i_bias; a.out = out; a.batch = batch; a.d_inner = d_inner;
  return launched(ss::launch_gated_step(a, dtype == SS_BF16, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------------------------ layer norm

static ss_status norm_sizes(int64_t rows, int64_t dim, int64_t* n) {
  if (rows < 0 || dim < 0)
    return fail(SS_ERR_INVALID_ARG, "negative size (rows=%lld dim=%lld)",
                static_cast<long long>(rows), static_cast<long long>(dim));
  if (dim > kMaxWidth)
    return fail(SS_ERR_UNSUPPORTED, "dim=%lld above 16777216", static_cast<long long>(dim));
  int64_t m;
  if (!mul_ok(rows, dim, n) || !mul_ok(*n, 64, &m))
    return fail(SS_ERR_INVALID_ARG, "sizes overflow 64-bit byte offsets");
  if (rows > kMaxGrid) return fail(SS_ERR_INVALID_ARG, "too many rows");
  return SS_OK;
}

ss_status ss_layer_norm_fwd(const void* x, const float* residual, const float* weight,
                            const float* bias, float eps, void* out, float* sum, float* mean,
                            float* rstd, int64_t rows, int64_t dim, ss_dtype dtype,
                            void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = norm_sizes(rows, dim, &n)) != SS_OK) return s;
  if (!(eps >= 0.0f) || isinf(eps))
    return fail(SS_ERR_INVALID_ARG, "eps=%g is not a finite number of at least 0",
                static_cast<double>(eps));
  if (n == 0) return ok();
  const Arr in[] = {{"x", x, n, es, true}, {"residual", residual, n, 4, false},
                    {"weight", weight, dim, 4, false}, {"bias", bias, dim, 4, false}};
  const Arr outs[] = {{"out", out, n, es, true}, {"sum", sum, n, 4, false},
                      {"mean", mean, rows, 4, false}, {"rstd", rstd, rows, 4, false}};
  if ((s = check_arrays(in, 4, outs, 4)) != SS_OK) return s;
  ss::NormArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.eps = eps; a.out = out;
  a.sum = sum; a.mean = mean; a.rstd = rstd; a.rows = rows; a.dim = dim;
  return launched(ss::launch_norm_fwd(a, dtype == SS_BF16, static_cast<hipStream_t>(stream)));
}

size_t ss_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  int64_t n;
  if (rows <= 0 || dim <= 0 || dim > kMaxWidth || rows > kMaxGrid || !mul_ok(rows, dim * 64, &n))
    return 0;
  return ss::norm_bwd_ws_bytes(rows, dim);
}

ss_status ss_layer_norm_bwd(const void* dout, const void* x, ss_dtype s_dtype,
                            const float* weight, const float* mean, const float* rstd,
                            const float* dsum, void* dx, float* dresidual, float* dweight,
                            float* dbias, int64_t rows, int64_t dim, ss_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  int64_t es = 0, ss_ = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = check_dtype(s_dtype, &ss_)) != SS_OK) return s;
  if (s_dtype != dtype && s_dtype != SS_F32)
    return fail(SS_ERR_UNSUPPORTED, "s is either of the io dtype or float32");
  if ((s = norm_sizes(rows, dim, &n)) != SS_OK) return s;
  if (dim == 0) return ok();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool some = n > 0;
  const size_t need = some && (dweight || dbias) ? ss::norm_bwd_ws_bytes(rows, dim) : 0;
  const Arr in[] = {{"dout", dout, n, es, some}, {"s", x, n, ss_, some},
                    {"weight", weight, dim, 4, false}, {"mean", mean, rows, 4, some},
                    {"rstd", rstd, rows, 4, some}, {"dsum", dsum, n, 4, false}};
  const Arr outs[] = {{"dx", dx, n, es, false}, {"dresidual", dresidual, n, 4, false},
                      {"dweight", dweight, dim, 4, false}, {"dbias", dbias, dim, 4, false},
                      {"workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1,
                       false}};
  if (some && !dx && !dresidual)
    return fail(SS_ERR_INVALID_ARG, "dx and dresidual are both NULL");
  if ((s = check_arrays(in, 6, outs, 5)) != SS_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "ss_layer_norm_bwd_workspace_bytes")) != SS_OK)
    return s;
  if (!some) {
    hipError_t e = hipSuccess;
    if (dweight) e = ss::launch_zero(dweight, dim, st);
    if (e == hipSuccess && dbias) e = ss::launch_zero(dbias, dim, st);
    return launched(e);
  }
  ss::NormArgs a{};
  a.dout = dout; a.x = x; a.s_f32 = s_dtype == SS_F32; a.weight = weight; a.mean_in = mean;
  a.rstd_in = rstd; a.dsum = dsum; a.dx = dx; a.dresidual = dresidual; a.dweight = dweight;
  a.dbias = dbias; a.workspace = workspace; a.rows = rows; a.dim = dim;
  return launched(ss::launch_norm_bwd(a, dtype == SS_BF16, st));
}

// ----------------------------------------------------------------------------------- convolution

// One wave per at least 16 steps and 64 channels, four to a workgroup.
static ss_status check_conv_grid(int64_t batch, int64_t seqlen, int64_t d_inner) {
  return check_grid((batch * ((seqlen + 15) / 16) + 3) / 4 * ((d_inner + 63) / 64), 256);
}

static ss_status check_width(int32_t k) {
  return k >= 1 && k <= 4 ? SS_OK : fail(SS_ERR_UNSUPPORTED, "k=%d outside 1..4", k);
}

ss_status ss_causal_conv_fwd(const void* x, const float* weight, const float* bias,
                             const void* x_prev, const uint8_t* starts, int silu, void* out,
                             int64_t batch, int64_t seqlen, int64_t d_inner, int32_t k,
                             ss_dtype dtype, void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = check_width(k)) != SS_OK) return s;
  if ((s = check_sizes(batch, seqlen, d_inner, &n)) != SS_OK) return s;
  if (n == 0) return ok();
  if ((s = check_conv_grid(batch, seqlen, d_inner)) != SS_OK) return s;
  const Arr in[] = {{"x", x, n, es, true}, {"weight", weight, d_inner * k, 4, true},
                    {"bias", bias, d_inner, 4, false},
                    {"x_prev", x_prev, batch * (k - 1) * d_inner, es, false},
                    {"starts", starts, batch * seqlen, 1, false}};
  const Arr outs[] = {{"out", out, n, es, true}};
  if ((s = check_arrays(in, 5, outs, 1)) != SS_OK) return s;
  ss::ConvArgs a{};
  a.x = x; a.weight = weight; a.bias = bias; a.x_prev = k > 1 ? x_prev : nullptr;
  a.starts = starts; a.out = out; a.batch = batch; a.seqlen = seqlen; a.d_inner = d_inner;
  a.k = k; a.silu = silu ? 1 : 0;
  return launched(ss::launch_conv_fwd(a, dtype == SS_BF16, static_cast<hipStream_t>(stream)));
}

size_t ss_causal_conv_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner,
                                          int32_t k, ss_dtype) {
  if (!sizes_ok(batch, seqlen, d_inner) || k < 1 || k > 4) return 0;
  return ss::conv_bwd_ws_bytes(batch, seqlen, d_inner, k);
}

ss_status ss_causal_conv_bwd(const void* x, const float* weight, const float* bias,
                             const void* x_prev, const uint8_t* starts, int silu,
                             const void* dout, void* dx, float* dweight, float* dbias,
                             void* dx_prev, int64_t batch, int64_t seqlen, int64_t d_inner,
                             int32_t k, ss_dtype dtype, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = check_width(k)) != SS_OK) return s;
  if ((s = check_sizes(batch, seqlen, d_inner, &n)) != SS_OK) return s;
  if (d_inner == 0) return ok();
  if ((s = check_conv_grid(batch, seqlen, d_inner)) != SS_OK) return s;
  const bool some = n > 0;
  const int64_t prev = batch * (k - 1) * d_inner;
  if (dx_prev && !x_prev && prev > 0)
    return fail(SS_ERR_INVALID_ARG, "dx_prev is given without x_prev");
  const size_t need = some ? ss::conv_bwd_ws_bytes(batch, seqlen, d_inner, k) : 0;
  const Arr in[] = {{"x", x, n, es, some}, {"weight", weight, d_inner * k, 4, true},
                    {"bias", bias, d_inner, 4, false}, {"x_prev", x_prev, prev, es, false},
                    {"starts", starts, batch * seqlen, 1, false}, {"dout", dout, n, es, some}};
  const Arr outs[] = {{"dx", dx, n, es, some}, {"dweight", dweight, d_inner * k, 4, true},
                      {"dbias", dbias, d_inner, 4, false}, {"dx_prev", dx_prev, prev, es, false},
                      {"workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1,
                       false}};
  if ((s = check_arrays(in, 6, outs, 5)) != SS_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "ss_causal_conv_bwd_workspace_bytes")) != SS_OK)
    return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  ss::ConvArgs a{};
  a.x = x; a.weight = weight; a.bias = bias; a.x_prev = k > 1 ? x_prev : nullptr;
  a.starts = starts; a.dout = dout; a.dx = dx; a.dweight = dweight; a.dbias = dbias;
  a.dx_prev = k > 1 ? dx_prev : nullptr; a.workspace = workspace; a.batch = batch;
  a.seqlen = seqlen; a.d_inner = d_inner; a.k = k; a.silu = silu ? 1 : 0;
  if (!some) {
    hipError_t e = ss::launch_zero(dweight, d_inner * k, st);
    if (e == hipSuccess && dbias) e = ss::launch_zero(dbias, d_inner, st);
    if (e == hipSuccess && a.dx_prev && prev)
      e = ss::launch_zero_bytes(a.dx_prev, prev * es, st);
    return launched(e);
  }
  return launched(ss::launch_conv_bwd(a, dtype == SS_BF16, st));
}

ss_status ss_causal_conv_update(void* conv_state, const void* x, const float* weight,
                                const float* bias, int silu, void* out, int64_t batch,
                                int64_t d_inner, int32_t k, ss_dtype dtype, void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = check_width(k)) != SS_OK) return s;
  if ((s = check_sizes(batch, 1, d_inner, &n)) != SS_OK) return s;
  if (n == 0) return ok();
  if ((s = check_grid((n + 255) / 256, 256)) != SS_OK) return s;
  const Arr in[] = {{"x", x, n, es, true}, {"weight", weight, d_inner * k, 4, true},
                    {"bias", bias, d_inner, 4, false}};
  const Arr outs[] = {{"conv_state", k > 1 ? conv_state : nullptr, batch * (k - 1) * d_inner, es,
                       k > 1},
                      {"out", out, n, es, true}};
  if ((s = check_arrays(in, 3, outs, 2)) != SS_OK) return s;
  ss::ConvArgs a{};
  a.x = x; a.weight = weight; a.bias = bias; a.conv_state = k > 1 ? conv_state : nullptr;
  a.out = out; a.batch = batch; a.seqlen = 1; a.d_inner = d_inner; a.k = k;
  a.silu = silu ? 1 : 0;
  return launched(ss::launch_conv_step(a, dtype == SS_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
