// api_checks.h -- what the entry points of the sequence and block operators have
// in common: refusals, launches counted before they are made, alignment, types,
// views, workspaces.
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "../../include/per_train.h"
#include "train_internal.h"

namespace per {

__attribute__((format(printf, 1, 2))) inline int bad(const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return api_fail(PER_EINVAL, buf);
}

// Runs a call's launches, once to count and then in earnest.
template <typename F>
int run(const char* what, F launch) {
  Launches& l = launches();
  l.counting = true;
  l.items = 0;
  hipError_t e = launch();
  l.counting = false;
  if (e == hipSuccess && l.items >> 32)
    return bad("%s would take %llu work-items in one launch, 2^32 or more: call it in pieces", what,
               (unsigned long long)l.items);
  if (e == hipSuccess) e = launch();
  if (e == hipSuccess) return api_ok();
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", what, hipGetErrorString(e));
  return api_fail(PER_EHIP, buf);
}

inline bool type_ok(int32_t t) { return t == PER_F32 || t == PER_BF16 || t == PER_F16; }
inline int size_of(int32_t t) { return t == PER_F32 ? 4 : 2; }

inline bool misaligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}

constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 40;

inline int check_view(const void* p, int32_t type, int64_t sb, int64_t st, const char* what) {
  if (!p) return bad("%s is required", what);
  if (misaligned(p, size_of(type))) return bad("%s is not aligned to its type", what);
  if (sb < 0 || st < 0 || sb > kMaxStride || st > kMaxStride)
    return bad("%s has a stride that is negative or too large", what);
  return PER_OK;
}

// An output's steps and sequences must not overlap: rows of D channels, the
// smaller stride's whole extent within the larger one.
inline int check_out_view(const void* p, int32_t type, int64_t B, int64_t T, int64_t D, int64_t sb,
                   int64_t st, const char* what) {
  const int rc = check_view(p, type, sb, st, what);
  if (rc) return rc;
  const bool t_inner = T <= 1 || (st >= D && (B <= 1 || sb >= (T - 1) * st + D));
  const bool b_inner = B <= 1 || (sb >= D && (T <= 1 || st >= (B - 1) * sb + D));
  if ((T <= 1 && B > 1 && sb < D) || !(t_inner || b_inner))
    return bad("%s has rows that overlap", what);
  return PER_OK;
}

inline int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return PER_OK;
  if (!ws) return bad("a workspace of %zu bytes is required", need);
  if (misaligned(ws, 16)) return bad("the workspace must be 16-byte aligned");
  if (have < need) {
    char buf[128];
    snprintf(buf, sizeof buf, "workspace of %zu bytes, %zu are needed", have, need);
    return api_fail(PER_ENOSPC, buf);
  }
  return PER_OK;
}

}  // namespace per
