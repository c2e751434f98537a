// ss_check.h -- argument checks that the C-ABI layers of the block operators share: arrays'
// presence, alignment and overlap, workspaces, launch sizes.
#pragma once

#include "ss_host.h"

namespace ss::host {

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
inline ss_status check_arrays(const Arr* in, int n_in, const Arr* out, int n_out) {
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

inline ss_status check_workspace(const void* ws, size_t have, size_t need, const char* query) {
  if (need == 0) return SS_OK;
  if (!ws || have < need)
    return fail(SS_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu bytes needed "
                "(%s)", ws ? have : size_t(0), need, query);
  if (!aligned(ws, 16))
    return fail(SS_ERR_UNSUPPORTED, "workspace pointer %p not 16-byte aligned", ws);
  return SS_OK;
}

inline ss_status launched(hipError_t e) {
  return e == hipSuccess ? ok() : fail(SS_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

// A launch counts its threads in 32 bits.
inline ss_status check_grid(int64_t blocks, int64_t threads) {
  if (blocks > 0xffffffffll / threads)
    return fail(SS_ERR_INVALID_ARG, "too many elements for one launch");
  return SS_OK;
}

}  // namespace ss::host
