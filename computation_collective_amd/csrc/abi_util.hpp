// Host-side helpers of the C entry points: error reporting and the argument
// checks they share.  Every check runs before anything is enqueued.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hocf.h"
#include "internal.hpp"

namespace hocf {

// Records the detail of this thread's error and returns its status; clears it.
hocf_status fail(hocf_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
hocf_status ok();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Checks on the sync block (no HIP call).  `need` = workspace bytes the call needs.
inline hocf_status check_sync(const hocf_sync* s, size_t need) {
  if (!s) return fail(HOCF_ERR_INVALID_ARG, "sync is NULL");
  if (s->epoch == 0) return fail(HOCF_ERR_INVALID_ARG, "epoch must be nonzero");
  if (need > 0) {
    if (!s->workspace) return fail(HOCF_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned16(s->workspace)) return fail(HOCF_ERR_INVALID_ARG, "workspace not 16-byte aligned");
    if (s->workspace_bytes < need)
      return fail(HOCF_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", s->workspace_bytes, need);
  }
  if (s->status && (reinterpret_cast<uintptr_t>(s->status) & 3u))
    return fail(HOCF_ERR_INVALID_ARG, "status word not 4-byte aligned");
  if (s->abort_flag && (reinterpret_cast<uintptr_t>(s->abort_flag) & 3u))
    return fail(HOCF_ERR_INVALID_ARG, "abort word not 4-byte aligned");
  return HOCF_OK;
}

// Converts a checked sync block for the kernels (queries the device clock).
inline hocf_status to_sync_args(const hocf_sync* s, SyncArgs* out) {
  DeviceInfo di;
  if (device_info(&di) != hipSuccess) return fail(HOCF_ERR_HIP, "device query failed");
  const uint64_t ns = s->spin_timeout_ns ? s->spin_timeout_ns : 1000000000ull;
  out->epoch = s->epoch;
  out->status = s->status;
  out->abort_flag = s->abort_flag;
  // wall_clock64() ticks at wall_clock_khz kHz
  const long double ticks = (long double)ns * (long double)di.wall_clock_khz / 1.0e6L;
  out->timeout_ticks = ticks > 1.8e19L ? ~0ull : (uint64_t)ticks;
  return HOCF_OK;
}

inline hocf_status check_windows(const hocf_window* win, int P, const char* what) {
  if (!win) return fail(HOCF_ERR_INVALID_ARG, "%s: window array is NULL", what);
  for (int r = 0; r < P; ++r) {
    if (!win[r].data || !win[r].flags)
      return fail(HOCF_ERR_INVALID_ARG, "%s: window %d has a NULL data or flags pointer", what, r);
    if (!aligned16(win[r].data) || (reinterpret_cast<uintptr_t>(win[r].flags) & 3u))
      return fail(HOCF_ERR_INVALID_ARG, "%s: window %d misaligned", what, r);
  }
  return HOCF_OK;
}

inline bool dt_ok(hocf_dtype d) { return d == HOCF_F32 || d == HOCF_BF16; }

// Byte ranges a call reads (inputs) and writes (outputs).  A written range
// may overlap no other range of the call: the kernels read their inputs
// while other workgroups already write, and publish into windows that others
// read, so any aliasing gives unspecified results.  Read-only ranges may
// overlap each other.  Empty ranges and NULL pointers are skipped.
class Ranges {
 public:
  void in(const char* what, int idx, const void* p, int64_t bytes) { add(what, idx, p, bytes, false); }
  void out(const char* what, int idx, const void* p, int64_t bytes) { add(what, idx, p, bytes, true); }
  hocf_status check(const char* op) const {
    for (int i = 0; i < n_; ++i)
      for (int j = i + 1; j < n_; ++j) {
        const R& a = r_[i];
        const R& b = r_[j];
        if (!a.out && !b.out) continue;
        if (a.lo < b.hi && b.lo < a.hi)
          return fail(HOCF_ERR_INVALID_ARG, "%s: %s[%d] and %s[%d] overlap (an output may alias nothing else)",
                      op, a.what, a.idx, b.what, b.idx);
      }
    return HOCF_OK;
  }

 private:
  struct R {
    const char* what;
    int idx;
    uintptr_t lo, hi;
    bool out;
  };
  void add(const char* what, int idx, const void* p, int64_t bytes, bool out) {
    if (!p || bytes <= 0 || n_ >= kMax) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    r_[n_++] = R{what, idx, lo, lo + (uintptr_t)bytes, out};
  }
  static constexpr int kMax = 4 * HOCF_MAX_P + 16;
  R r_[kMax];
  int n_ = 0;
};

// The sync block's own ranges: the status word and the workspace (both written).
inline void add_sync(Ranges& rg, const hocf_sync* s, size_t ws_bytes) {
  rg.out("status", 0, s->status, 4);
  rg.out("workspace", 0, s->workspace, (int64_t)ws_bytes);
}

inline hocf_status launched(int e, const char* what) {
  if (e == kNoKernel) return fail(HOCF_ERR_UNSUPPORTED, "%s: no kernel for this shape", what);
  if (e != hipSuccess) return fail(HOCF_ERR_HIP, "%s: %s", what, hipGetErrorString(static_cast<hipError_t>(e)));
  return ok();
}

}  // namespace hocf
