// zero_host.h -- what the host sources of libzero.so share: the plan, the
// calling thread's error text and the argument checks.
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <string>
#include <vector>

#include "zero.h"
#include "zero_internal.h"

struct zero_plan_s {
  int64_t psi = 0;
  int32_t n_d = 1;
  int64_t bucket_cap = 0;
  int32_t align = 1;
  int64_t psi_pad = 0;
  int64_t shard_total = 0;
  struct Bucket {
    int64_t flat_off, numel, padded, shard_numel, shard_off;
  };
  std::vector<Bucket> buckets;
  std::vector<int64_t> t_numel;
  std::vector<int64_t> t_off;
  std::vector<int32_t> t_bucket;
};

namespace zk {
namespace host {

// Text of the calling thread's last failure.
inline thread_local std::string g_err;

inline zero_status fail(zero_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

inline zero_status ok() { return ZERO_OK; }

inline int esize(int dt) { return dt == ZERO_F32 ? 4 : 2; }
inline bool is16(int dt) { return dt == ZERO_F16 || dt == ZERO_BF16; }
inline bool valid_dt(int dt) { return dt == ZERO_F32 || dt == ZERO_F16 || dt == ZERO_BF16; }

struct Range {
  uint64_t lo, hi;  // [lo, hi) bytes
  const char* what;
};

inline Range range_of(const void* p, int64_t elems, int es, const char* what) {
  const uint64_t lo = (uint64_t)(uintptr_t)p;
  return Range{lo, lo + (uint64_t)elems * (uint64_t)es, what};
}

inline bool overlap(const Range& a, const Range& b) {
  if (a.hi == a.lo || b.hi == b.lo) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned(const void* p, int bytes) { return ((uintptr_t)p % (uintptr_t)bytes) == 0; }

inline zero_status hip_fail(int err) {
  return fail(ZERO_EHIP, "HIP launch failed: %s (%d)", zk::hip_error_string(err), err);
}

inline zero_status check_plan(zero_plan_t p) {
  if (!p) return fail(ZERO_EINVAL, "plan is NULL");
  return ok();
}

}  // namespace host
}  // namespace zk
