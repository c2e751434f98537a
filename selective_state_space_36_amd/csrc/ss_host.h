// ss_host.h -- host-side helpers shared by the C-ABI translation units: status and message,
// overflow-checked products, pointer ranges and alignment.  Nothing here allocates or throws.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ss_scan.h"

namespace ss::host {

// Sets the calling thread's message (ss_last_error) and returns `s`; ok() clears it.
ss_status fail(ss_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ss_status ok();

inline bool mul_ok(int64_t a, int64_t b, int64_t* r) { return !__builtin_mul_overflow(a, b, r); }

struct Range {
  const char* name;
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range(const char* name, const void* p, int64_t elems, int64_t esize) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{name, lo, p ? lo + static_cast<uintptr_t>(elems * esize) : lo};
}

inline bool overlap(const Range& a, const Range& b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned(const void* p, int64_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline ss_status check_dtype(ss_dtype dt, int64_t* esize) {
  if (dt == SS_F32) { *esize = 4; return SS_OK; }
  if (dt == SS_BF16) { *esize = 2; return SS_OK; }
  return fail(SS_ERR_UNSUPPORTED, "unknown dtype %d", static_cast<int>(dt));
}

}  // namespace ss::host
