// ss_head_api.hip -- the C ABI of the operators around the multi-head scan (declared in
// include/ss_scan.h): argument checking, workspace sizes and dispatch.  No allocation, no
// synchronisation, no printing, nothing that throws.
#include <math.h>

#include "ss_check.h"
#include "ss_head.h"

namespace {

using namespace ss::host;

// Elements from the first to the last of `rows` rows of `width`, `stride` apart.
int64_t span(int64_t rows, int64_t stride, int64_t width) {
  return rows > 0 && width > 0 ? (rows - 1) * stride + width : 0;
}

ss_status check_stride(const char* name, int64_t rows, int64_t stride, int64_t width) {
  int64_t n;
  if (stride < width)
    return fail(SS_ERR_INVALID_ARG, "%s_stride=%lld below the row's %lld elements", name,
                static_cast<long long>(stride), static_cast<long long>(width));
  if (!mul_ok(rows, stride, &n) || !mul_ok(n, 64, &n))
    return fail(SS_ERR_INVALID_ARG, "sizes overflow 64-bit byte offsets");
  return SS_OK;
}

// ------------------------------------------------------------------------- the multi-head scan

struct HeadSizes {
  int64_t heads = 0, elems = 0, dts = 0, bcs = 0, states = 0, chunks = 0;
};

ss_status head_sizes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                     int64_t ngroups, int64_t d_state, HeadSizes* z) {
  if (batch < 0 || seqlen < 0 || nheads < 0 || headdim < 0 || ngroups < 0 || d_state < 0)
    return fail(SS_ERR_INVALID_ARG, "negative size");
  if (d_state < 1 || d_state > 256)
    return fail(SS_ERR_UNSUPPORTED, "d_state=%lld outside 1..256",
                static_cast<long long>(d_state));
  if (nheads > 0 && (ngroups < 1 || nheads % ngroups != 0))
    return fail(SS_ERR_INVALID_ARG, "nheads=%lld is not a multiple of ngroups=%lld",
                static_cast<long long>(nheads), static_cast<long long>(ngroups));
  if (headdim > kMaxWidth || nheads > kMaxWidth || seqlen > kMaxSteps)
    return fail(SS_ERR_UNSUPPORTED, "headdim or nheads above 16777216, or seqlen above "
                "2147483647");
  z->chunks = (seqlen + ss::kScan2BwdChunk - 1) / ss::kScan2BwdChunk;
  int64_t n, m;
  if (!mul_ok(batch, nheads, &z->heads) || !mul_ok(z->heads, seqlen, &z->dts) ||
      !mul_ok(z->dts, headdim, &z->elems) || !mul_ok(batch, ngroups, &z->bcs) ||
      !mul_ok(z->bcs, seqlen, &z->bcs) || !mul_ok(z->bcs, d_state, &z->bcs) ||
      !mul_ok(z->heads, d_state * headdim, &z->states) ||
      !mul_ok(z->states, z->chunks + 1, &n) || !mul_ok(n, 64, &m) || !mul_ok(z->elems, 64, &m) ||
      !mul_ok(z->bcs, 64, &n) || !mul_ok(n, nheads > 0 ? nheads : 1, &m))
    return fail(SS_ERR_INVALID_ARG, "sizes overflow 64-bit byte offsets");
  return SS_OK;
}

}  // namespace

extern "C" {

size_t ss_scan2_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads,
                                    int64_t headdim, int64_t ngroups, int64_t d_state,
                                    ss_dtype) {
  HeadSizes z;
  if (head_sizes(batch, seqlen, nheads, headdim, ngroups, d_state, &z) != SS_OK) return 0;
  if (z.elems == 0) return 0;
  return static_cast<size_t>(ss::scan2_bwd_ws_floats(batch, seqlen, nheads, headdim, ngroups,
                                                     d_state, nullptr, nullptr)) *
         sizeof(float);
}

ss_status ss_scan2_bwd(const void* x, const void* dt, const float* A, const void* B,
                       const void* C, const float* D, const void* z, const float* dt_bias,
                       int dt_softplus, const float* h0, const void* dout, const float* dh_last,
                       void* dx, void* ddt, void* dz, float* dA, void* dB, void* dC, float* dD,
                       float* ddt_bias, float* dh0, int64_t batch, int64_t seqlen,
                       int64_t nheads, int64_t headdim, int64_t ngroups, int64_t d_state,
                       ss_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t es = 0;
  HeadSizes n;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = head_sizes(batch, seqlen, nheads, headdim, ngroups, d_state, &n)) != SS_OK) return s;
  if (nheads == 0) return ok();
  const bool some = n.elems > 0;
  ss::Scan2BwdArgs a{};
  a.x = x; a.dt = dt; a.z = z; a.B = B; a.C = C; a.dout = dout; a.A = A; a.D = D;
  a.dt_bias = dt_bias; a.h0 = h0; a.dh_last = dh_last; a.dx = dx; a.ddt = ddt; a.dz = dz;
  a.dB = dB; a.dC = dC; a.dA = dA; a.dD = dD; a.ddt_bias = ddt_bias; a.dh0 = dh0;
  a.batch = batch; a.seqlen = seqlen; a.nheads = nheads; a.ngroups = ngroups;
  a.headdim = static_cast<int32_t>(headdim); a.d_state = static_cast<int32_t>(d_state);
  a.softplus = dt_softplus ? 1 : 0;
  const size_t need =
      some ? static_cast<size_t>(ss::scan2_bwd_ws_floats(batch, seqlen, nheads, headdim, ngroups,
                                                         d_state, &a,
                                                         static_cast<float*>(workspace))) *
                 sizeof(float)
           : 0;
  if (some) {
    if ((s = check_grid(2 * n.heads * a.n_pblk * (a.cut ? n.chunks : 1), 512)) != SS_OK) return s;
    if ((s = check_grid(batch * n.chunks * ngroups * a.splits, 512)) != SS_OK) return s;
  }
  const Arr in[] = {{"x", x, n.elems, es, some}, {"dt", dt, n.dts, es, some},
                    {"A", A, nheads, 4, true}, {"B", B, n.bcs, es, some},
                    {"C", C, n.bcs, es, some}, {"D", D, nheads, 4, false},
                    {"z", z, n.elems, es, false}, {"dt_bias", dt_bias, nheads, 4, false},
                    {"h0", h0, n.states, 4, false}, {"dout", dout, n.elems, es, some},
                    {"dh_last", dh_last, n.states, 4, false}};
  const Arr outs[] = {{"dx", dx, n.elems, es, some}, {"ddt", ddt, n.dts, es, some},
                      {"dz", z ? dz : nullptr, n.elems, es, some && z},
                      {"dA", dA, nheads, 4, true}, {"dB", dB, n.bcs, es, some},
                      {"dC", dC, n.bcs, es, some}, {"dD", dD, nheads, 4, false},
                      {"ddt_bias", ddt_bias, nheads, 4, false},
                      {"dh0", dh0, n.states, 4, false},
                      {"workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1,
                       false}};
  if ((s = check_arrays(in, 11, outs, 10)) != SS_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, need, "ss_scan2_bwd_workspace_bytes")) !=
      SS_OK)
    return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (!some) {  // no token: the sums are 0, what arrives behind the last step arrives before it
    hipError_t e = ss::launch_zero(dA, nheads, st);
    if (e == hipSuccess && dD) e = ss::launch_zero(dD, nheads, st);
    if (e == hipSuccess && ddt_bias) e = ss::launch_zero(ddt_bias, nheads, st);
    if (e == hipSuccess && dh0 && n.states)
      e = dh_last ? ss::launch_copy(dh0, dh_last, n.states, st)
                  : ss::launch_zero(dh0, n.states, st);
    // without channels the tokens' other gradients are 0 as well
    if (e == hipSuccess && ddt && n.dts) e = ss::launch_zero_bytes(ddt, n.dts * es, st);
    if (e == hipSuccess && dB && n.bcs) e = ss::launch_zero_bytes(dB, n.bcs * es, st);
    if (e == hipSuccess && dC && n.bcs) e = ss::launch_zero_bytes(dC, n.bcs * es, st);
    return launched(e);
  }
  return launched(ss::launch_scan2_bwd(a, dtype == SS_BF16, st));
}

ss_status ss_scan2_state_update(float* state, const void* x, const void* dt, const float* A,
                                const void* B, const void* C, const float* D, const void* z,
                                const float* dt_bias, int dt_softplus, void* out, int64_t batch,
                                int64_t nheads, int64_t headdim, int64_t ngroups,
                                int64_t d_state, ss_dtype dtype, void* stream) {
  int64_t es = 0;
  HeadSizes n;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = head_sizes(batch, 1, nheads, headdim, ngroups, d_state, &n)) != SS_OK) return s;
  if (n.elems == 0) return ok();
  if ((s = check_grid(n.heads * ((headdim + 15) / 16), 256)) != SS_OK) return s;
  const Arr in[] = {{"x", x, n.elems, es, true}, {"dt", dt, n.dts, es, true},
                    {"A", A, nheads, 4, true}, {"B", B, n.bcs, es, true},
                    {"C", C, n.bcs, es, true}, {"D", D, nheads, 4, false},
                    {"z", z, n.elems, es, false}, {"dt_bias", dt_bias, nheads, 4, false}};
  const Arr outs[] = {{"state", state, n.states, 4, true}, {"out", out, n.elems, es, true}};
  if ((s = check_arrays(in, 8, outs, 2)) != SS_OK) return s;
  ss::Scan2StepArgs a{};
  a.state = state; a.x = x; a.dt = dt; a.z = z; a.B = B; a.C = C; a.A = A; a.D = D;
  a.dt_bias = dt_bias; a.out = out; a.x_stride = a.z_stride = nheads * headdim;
  a.dt_stride = nheads; a.b_stride = a.c_stride = ngroups * d_state;
  a.softplus = dt_softplus ? 1 : 0; a.headdim = static_cast<int32_t>(headdim);
  a.d_state = static_cast<int32_t>(d_state); a.batch = batch; a.nheads = nheads;
  a.ngroups = ngroups;
  return launched(ss::launch_scan2_step(a, dtype == SS_BF16, static_cast<hipStream_t>(stream)));
}

size_t ss_scan2_state_update_conv_workspace_bytes(int64_t batch, int64_t nheads, int64_t headdim,
                                                  int64_t ngroups, int64_t d_state) {
  HeadSizes z;
  if (head_sizes(batch, 1, nheads, headdim, ngroups, d_state, &z) != SS_OK) return 0;
  return static_cast<size_t>(z.elems ? z.elems + 2 * z.bcs : 0) * sizeof(float);
}

ss_status ss_scan2_state_update_conv(float* state, void* conv_state, const void* xbc,
                                     int64_t xbc_stride, const float* conv_weight,
                                     const float* conv_bias, int32_t conv_k, const void* dt,
                                     int64_t dt_stride, const float* A, const float* D,
                                     const void* z, int64_t z_stride, const float* dt_bias,
                                     int dt_softplus, void* out, int64_t batch, int64_t nheads,
                                     int64_t headdim, int64_t ngroups, int64_t d_state,
                                     ss_dtype dtype, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  int64_t es = 0;
  HeadSizes n;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if (conv_k < 1 || conv_k > 4)
    return fail(SS_ERR_UNSUPPORTED, "conv_k=%d outside 1..4", conv_k);
  if ((s = head_sizes(batch, 1, nheads, headdim, ngroups, d_state, &n)) != SS_OK) return s;
  if (n.elems == 0) return ok();
  const int64_t d = nheads * headdim, width = d + 2 * ngroups * d_state;
  if ((s = check_stride("xbc", batch, xbc_stride, width)) != SS_OK) return s;
  if ((s = check_stride("dt", batch, dt_stride, nheads)) != SS_OK) return s;
  if (z && (s = check_stride("z", batch, z_stride, d)) != SS_OK) return s;
  if ((s = check_grid(n.heads * ((headdim + 15) / 16), 256)) != SS_OK) return s;
  if ((s = check_grid((batch * width + 255) / 256, 256)) != SS_OK) return s;
  const int64_t need = batch * width * 4;
  const Arr in[] = {{"xbc", xbc, span(batch, xbc_stride, width), es, true},
                    {"conv_weight", conv_weight, width * conv_k, 4, true},
                    {"conv_bias", conv_bias, width, 4, false},
                    {"dt", dt, span(batch, dt_stride, nheads), es, true},
                    {"A", A, nheads, 4, true}, {"D", D, nheads, 4, false},
                    {"z", z, z ? span(batch, z_stride, d) : 0, es, false},
                    {"dt_bias", dt_bias, nheads, 4, false}};
  const Arr outs[] = {{"state", state, n.states, 4, true},
                      {"conv_state", conv_k > 1 ? conv_state : nullptr,
                       batch * (conv_k - 1) * width, es, conv_k > 1},
                      {"out", out, n.elems, es, true},
                      {"workspace", workspace, workspace ? need : 0, 1, false}};
  if ((s = check_arrays(in, 8, outs, 4)) != SS_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, static_cast<size_t>(need),
                           "ss_scan2_state_update_conv_workspace_bytes")) != SS_OK)
    return s;
  ss::Scan2StepArgs a{};
  a.act = static_cast<float*>(workspace);
  a.state = state; a.x = a.act; a.B = a.act + d; a.C = a.act + d + ngroups * d_state;
  a.x_stride = a.b_stride = a.c_stride = a.conv_dim = width;
  a.dt = dt; a.dt_stride = dt_stride; a.z = z; a.z_stride = z_stride; a.A = A; a.D = D;
  a.dt_bias = dt_bias; a.out = out; a.conv_state = conv_state; a.xbc = xbc;
  a.xbc_stride = xbc_stride; a.conv_weight = conv_weight; a.conv_bias = conv_bias;
  a.conv_k = conv_k; a.softplus = dt_softplus ? 1 : 0;
  a.headdim = static_cast<int32_t>(headdim); a.d_state = static_cast<int32_t>(d_state);
  a.batch = batch; a.nheads = nheads; a.ngroups = ngroups;
  return launched(ss::launch_scan2_step(a, dtype == SS_BF16, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------------------ norms, dropout

static ss_status rows_sizes(int64_t rows, int64_t dim, int64_t* n) {
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

static ss_status check_eps(float eps) {
  if (!(eps >= 0.0f) || isinf(eps))
    return fail(SS_ERR_INVALID_ARG, "eps=%g is not a finite number of at least 0",
                static_cast<double>(eps));
  return SS_OK;
}

// p in 2^-16 parts; without any nothing is dropped and rng is not read.
static ss_status check_drop(double p, const uint64_t* rng, ss::DropArgs* d) {
  if (!(p >= 0.0 && p <= 1.0))
    return fail(SS_ERR_INVALID_ARG, "p=%g is not a probability", p);
  const double cut = rint(p * 65536.0);
  *d = ss::DropArgs{nullptr, 0, 1.0f};
  if (cut == 0.0) return SS_OK;
  if (!rng) return fail(SS_ERR_INVALID_ARG, "rng is NULL");
  if (!aligned(rng, 8))
    return fail(SS_ERR_UNSUPPORTED, "rng pointer %p not aligned to its 8-byte element",
                static_cast<const void*>(rng));
  d->rng = rng;
  d->cut = static_cast<uint32_t>(cut);
  d->up = cut < 65536.0 ? static_cast<float>(65536.0 / (65536.0 - cut)) : 0.0f;
  return SS_OK;
}

ss_status ss_rms_norm_fwd(const void* x, const float* residual, const float* weight,
                          const float* scale, int norm_branch, double p, const uint64_t* rng,
                          float eps, void* out, float* sum, float* rstd, float* branch_rstd,
                          int64_t rows, int64_t dim, ss_dtype dtype, void* stream) {
  int64_t es = 0, n = 0;
  ss::RmsArgs a{};
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = rows_sizes(rows, dim, &n)) != SS_OK) return s;
  if ((s = check_eps(eps)) != SS_OK) return s;
  if ((s = check_drop(p, rng, &a.drop)) != SS_OK) return s;
  if (n == 0) return ok();
  const Arr in[] = {{"x", x, n, es, true}, {"residual", residual, n, 4, false},
                    {"weight", weight, dim, 4, false}, {"scale", scale, dim, 4, false},
                    {"rng", a.drop.rng, 2, 8, false}};
  const Arr outs[] = {{"out", out, n, es, true}, {"sum", sum, n, 4, false},
                      {"rstd", rstd, rows, 4, false},
                      {"branch_rstd", branch_rstd, rows, 4, false}};
  if ((s = check_arrays(in, 5, outs, 4)) != SS_OK) return s;
  a.x = x; a.residual = residual; a.weight = weight; a.scale = scale;
  a.branch = norm_branch != 0; a.eps = eps; a.out = out; a.sum = sum; a.rstd = rstd;
  a.branch_rstd = branch_rstd; a.rows = rows; a.dim = dim;
  return launched(ss::launch_rms_fwd(a, dtype == SS_BF16, static_cast<hipStream_t>(stream)));
}

size_t ss_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  int64_t n;
  if (rows_sizes(rows, dim, &n) != SS_OK || n == 0) return 0;
  return ss::rms_bwd_ws_bytes(rows, dim);
}

ss_status ss_rms_norm_bwd(const void* dout, const void* sum, ss_dtype s_dtype,
                          const float* weight, const float* rstd, const void* x,
                          const float* scale, int norm_branch, const float* branch_rstd,
                          double p, const uint64_t* rng, const float* dsum, void* dx,
                          float* dresidual, float* dweight, float* dscale, int64_t rows,
                          int64_t dim, ss_dtype dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int64_t es = 0, ses = 0, n = 0;
  ss::RmsArgs a{};
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = check_dtype(s_dtype, &ses)) != SS_OK) return s;
  if (s_dtype != dtype && s_dtype != SS_F32)
    return fail(SS_ERR_UNSUPPORTED, "s is either of the io dtype or float32");
  if ((s = rows_sizes(rows, dim, &n)) != SS_OK) return s;
  if ((s = check_drop(p, rng, &a.drop)) != SS_OK) return s;
  if (dim == 0) return ok();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool some = n > 0, branch = norm_branch != 0;
  if (s_dtype != SS_F32 && (branch || scale || a.drop.rng))
    return fail(SS_ERR_INVALID_ARG, "s has to be the float32 sum with scale, norm_branch or "
                "dropout");
  const size_t need = some && (dweight || dscale) ? ss::rms_bwd_ws_bytes(rows, dim) : 0;
  const bool want_x = branch || dscale;
  const Arr in[] = {{"dout", dout, n, es, some}, {"s", sum, n, ses, some},
                    {"weight", weight, dim, 4, false}, {"rstd", rstd, rows, 4, some},
                    {"x", want_x ? x : nullptr, n, es, some && want_x},
                    {"scale", scale, dim, 4, false},
                    {"branch_rstd", branch ? branch_rstd : nullptr, rows, 4, some && branch},
                    {"rng", a.drop.rng, 2, 8, false}, {"dsum", dsum, n, 4, false}};
  const Arr outs[] = {{"dx", dx, n, es, false}, {"dresidual", dresidual, n, 4, false},
                      {"dweight", dweight, dim, 4, false}, {"dscale", dscale, dim, 4, false},
                      {"workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1,
                       false}};
  if (some && !dx && !dresidual)
    return fail(SS_ERR_INVALID_ARG, "dx and dresidual are both NULL");
  if ((s = check_arrays(in, 9, outs, 5)) != SS_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "ss_rms_norm_bwd_workspace_bytes")) != SS_OK)
    return s;
  if (!some) {
    hipError_t e = hipSuccess;
    if (dweight) e = ss::launch_zero(dweight, dim, st);
    if (e == hipSuccess && dscale) e = ss::launch_zero(dscale, dim, st);
    return launched(e);
  }
  a.dout = dout; a.s = sum; a.s_f32 = s_dtype == SS_F32; a.weight = weight; a.rstd_in = rstd;
  a.x = want_x ? x : nullptr; a.scale = scale; a.branch = branch; a.branch_rstd_in = branch_rstd;
  a.dsum = dsum; a.dx = dx; a.dresidual = dresidual; a.dweight = dweight; a.dscale = dscale;
  a.workspace = static_cast<float*>(workspace); a.rows = rows; a.dim = dim;
  return launched(ss::launch_rms_bwd(a, dtype == SS_BF16, st));
}

static ss_status check_groups(int64_t rows, int64_t dim, int64_t groups) {
  if (groups < 1 || dim % groups != 0)
    return fail(SS_ERR_INVALID_ARG, "dim=%lld is not a multiple of groups=%lld",
                static_cast<long long>(dim), static_cast<long long>(groups));
  // rows * groups, and the workgroups of the backward, whose number is a multiple of the groups
  if (groups > (int64_t(1) << 20) || rows * groups > kMaxGrid)
    return fail(SS_ERR_INVALID_ARG, "too many groups");
  return SS_OK;
}

ss_status ss_gated_norm_fwd(const void* x, const void* z, int64_t z_stride, const float* weight,
                            int gate_first, float eps, void* out, float* rstd, int64_t rows,
                            int64_t dim, int64_t groups, ss_dtype dtype, void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = rows_sizes(rows, dim, &n)) != SS_OK) return s;
  if ((s = check_eps(eps)) != SS_OK) return s;
  if ((s = check_groups(rows, dim, groups)) != SS_OK) return s;
  if (n == 0) return ok();
  if (z && (s = check_stride("z", rows, z_stride, dim)) != SS_OK) return s;
  const Arr in[] = {{"x", x, n, es, true}, {"z", z, z ? span(rows, z_stride, dim) : 0, es, false},
                    {"weight", weight, dim, 4, false}};
  const Arr outs[] = {{"out", out, n, es, true}, {"rstd", rstd, rows * groups, 4, false}};
  if ((s = check_arrays(in, 3, outs, 2)) != SS_OK) return s;
  ss::GatedNormArgs a{};
  a.x = x; a.z = z; a.z_stride = z_stride; a.weight = weight; a.gate_first = gate_first != 0;
  a.eps = eps; a.out = out; a.rstd = rstd; a.rows = rows; a.dim = dim; a.groups = groups;
  return launched(
      ss::launch_gated_norm_fwd(a, dtype == SS_BF16, static_cast<hipStream_t>(stream)));
}

size_t ss_gated_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t groups) {
  int64_t n;
  if (rows_sizes(rows, dim, &n) != SS_OK || n == 0 || check_groups(rows, dim, groups) != SS_OK)
    return 0;
  return ss::gated_norm_bwd_ws_bytes(rows, dim, groups);
}

ss_status ss_gated_norm_bwd(const void* dout, const void* x, const void* z, int64_t z_stride,
                            const float* weight, const float* rstd, int gate_first, void* dx,
                            void* dz, float* dweight, int64_t rows, int64_t dim, int64_t groups,
                            ss_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
  int64_t es = 0, n = 0;
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = rows_sizes(rows, dim, &n)) != SS_OK) return s;
  if ((s = check_groups(rows, dim, groups)) != SS_OK) return s;
  if (dim == 0) return ok();
  const bool some = n > 0;
  if (z && (s = check_stride("z", rows, z_stride, dim)) != SS_OK) return s;
  const size_t need = some && dweight ? ss::gated_norm_bwd_ws_bytes(rows, dim, groups) : 0;
  const Arr in[] = {{"dout", dout, n, es, some}, {"x", x, n, es, some},
                    {"z", z, z ? span(rows, z_stride, dim) : 0, es, false},
                    {"weight", weight, dim, 4, false}, {"rstd", rstd, rows * groups, 4, some}};
  const Arr outs[] = {{"dx", dx, n, es, some}, {"dz", z ? dz : nullptr, n, es, some && z},
                      {"dweight", dweight, dim, 4, false},
                      {"workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1,
                       false}};
  if ((s = check_arrays(in, 5, outs, 4)) != SS_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "ss_gated_norm_bwd_workspace_bytes")) != SS_OK)
    return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (!some) return launched(dweight ? ss::launch_zero(dweight, dim, st) : hipSuccess);
  ss::GatedNormArgs a{};
  a.dout = dout; a.x = x; a.z = z; a.z_stride = z_stride; a.weight = weight; a.rstd_in = rstd;
  a.gate_first = gate_first != 0; a.dx = dx; a.dz = dz; a.dweight = dweight;
  a.workspace = static_cast<float*>(workspace); a.rows = rows; a.dim = dim; a.groups = groups;
  return launched(ss::launch_gated_norm_bwd(a, dtype == SS_BF16, st));
}

ss_status ss_dropout(const void* x, void* out, double p, const uint64_t* rng, int64_t rows,
                     int64_t dim, ss_dtype dtype, void* stream) {
  int64_t es = 0, n = 0;
  ss::DropArgs d{};
  ss_status s = check_dtype(dtype, &es);
  if (s != SS_OK) return s;
  if ((s = rows_sizes(rows, dim, &n)) != SS_OK) return s;
  if (!rng) return fail(SS_ERR_INVALID_ARG, "rng is NULL");
  if ((s = check_drop(p, rng, &d)) != SS_OK) return s;
  if (n == 0) return ok();
  d.rng = rng;  // with nothing to drop the call is a copy
  const Arr in[] = {{"x", x, n, es, true}, {"rng", rng, 2, 8, true}};
  const Arr outs[] = {{"out", out, n, es, true}};
  if ((s = check_arrays(in, 2, outs, 1)) != SS_OK) return s;
  return launched(ss::launch_dropout(x, out, d, rows, dim, dtype == SS_BF16,
                                     static_cast<hipStream_t>(stream)));
}

}  // extern "C"
