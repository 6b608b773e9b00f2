// The argument validation of the mixture-of-experts entries, built with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host code by
// tests/test_sanitize_moe_cpu.py: every integer argument at the ends of its
// type and around its limits, alone and against one other argument's.  Every
// call is to fail: the sync block is invalid (the arithmetic of the checks
// before it), or all tensors are one (the sizes of the ranges).  The pointers
// are fake addresses, never dereferenced.  Exit status 0 when every call
// returned an error, or HOCF_OK for a call with nothing to do.
#include <climits>
#include <cstdint>
#include <cstdio>

#include "hocf.h"

static const int64_t kEnds[] = {INT64_MIN, INT64_MAX, INT_MIN, INT_MAX, -1, 0, 1, 2, 7, 8, 16, 17, 32, 64, 128, 512, 1024,
                                1 << 20, (1 << 20) + 8, 1 << 24, int64_t(1) << 31, (int64_t(1) << 31) - 8, int64_t(1) << 40};
static long calls = 0, unexpected = 0;

// Calls fn on the base arguments with every end in every place, and in every pair of places.
template <int N, class FN>
static void sweep(const char* name, const int64_t (&base)[N], FN fn) {
  auto one = [&](const int64_t (&a)[N]) {
    const hocf_status st = fn(a);
    ++calls;
    if (st == HOCF_ERR_HIP || (int)st < 0 || (int)st > HOCF_ERR_CAPACITY) {
      if (++unexpected <= 10) std::fprintf(stderr, "%s: status %d (%s)\n", name, (int)st, hocf_last_error());
    }
  };
  for (int i = 0; i < N; ++i)
    for (int64_t u : kEnds)
      for (int j = i; j < N; ++j)
        for (int64_t v : kEnds) {
          int64_t a[N];
          for (int k = 0; k < N; ++k) a[k] = base[k];
          a[i] = u;
          if (j > i) a[j] = v;
          one(a);
          if (j == i) break;
        }
}

int main() {
  char* const p = reinterpret_cast<char*>(uintptr_t(1) << 44);
  int32_t* const i32 = reinterpret_cast<int32_t*>(p);
  int64_t* const i64 = reinterpret_cast<int64_t*>(p);
  float* const f = reinterpret_cast<float*>(p);
  uint32_t* const u32 = reinterpret_cast<uint32_t*>(p);
  uint8_t* const u8 = reinterpret_cast<uint8_t*>(p);
  hocf_sync one{};  // (its workspace is the tensors' memory too)
  one.epoch = 1;
  one.workspace = p;
  one.workspace_bytes = size_t(1) << 40;
  one.status = u32;
  hocf_sync bad = one;
  bad.epoch = 0;
  const hocf_sync* syncs[] = {&bad, &one};
  auto dt = [](int64_t v) { return static_cast<hocf_dtype>((int)v); };

  for (const hocf_sync* s : syncs) {
    sweep("moe_route", {100, 64, 4, HOCF_F32, 64, 0, 8, 4, 2, 1}, [&](const int64_t(&a)[10]) {
      return hocf_moe_route(a[0], (int)a[1], (int)a[2], dt(a[3]), p, a[4], f, static_cast<hocf_score>((int)a[5]), (int)a[6],
                            (int)a[7], (int)a[8], (int)a[9], 1.0f, i32, f, i32, s, nullptr);
    });
    sweep("moe_route_bwd", {100, 64, 4, HOCF_BF16, 64, 1, 1}, [&](const int64_t(&a)[7]) {
      return hocf_moe_route_bwd(a[0], (int)a[1], (int)a[2], dt(a[3]), p, a[4], i32, f, static_cast<hocf_score>((int)a[5]),
                                (int)a[6], 1.0f, p, s, nullptr);
    });
    sweep("moe_slots", {100, 2, 4, 2, 64}, [&](const int64_t(&a)[5]) {
      return hocf_moe_slots(a[0], (int)a[1], (int)a[2], (int)a[3], a[4], i32, i32, i32, i64, s, nullptr);
    });
    for (int32_t* index : {i32, (int32_t*)nullptr}) {
      sweep("moe_combine", {100, 2, 64, 200, HOCF_BF16, HOCF_F32}, [&](const int64_t(&a)[6]) {
        return hocf_moe_combine(a[0], (int)a[1], (int)a[2], a[3], dt(a[4]), dt(a[5]), p, f, index, p, p, s, nullptr);
      });
      sweep("moe_combine_bwd", {100, 2, 64, 200, HOCF_BF16, HOCF_F32}, [&](const int64_t(&a)[6]) {
        return hocf_moe_combine_bwd(a[0], (int)a[1], (int)a[2], a[3], dt(a[4]), dt(a[5]), p, f, p, index, index, p, f, s,
                                    nullptr);
      });
    }
    for (int64_t K : {256, 1 << 20})
      sweep("gemv_w4", {8, 2, 4, 0, 64, K, 64, HOCF_F32}, [&](const int64_t(&a)[8]) {
        return hocf_gemv_w4((int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)a[4], (int)a[5], (int)a[6], dt(a[7]), p, i32,
                            u32, p, p, p, s, nullptr);
      });
  }
  for (int64_t K : {256, 1 << 20})
    sweep("w4_pack", {2, 64, K, 64}, [&](const int64_t(&a)[4]) {
      return hocf_w4_pack((int)a[0], (int)a[1], (int)a[2], (int)a[3], u8, p, p, u32, p, p, nullptr);
    });
  for (int64_t a : kEnds) {
    (void)hocf_moe_route_workspace_bytes((int)a);
    for (int64_t b : kEnds)
      for (int64_t c : kEnds) (void)hocf_moe_slots_workspace_bytes(a, (int)b, (int)c);
  }
  std::printf("moe abi driver: %ld calls, %ld failures\n", calls, unexpected);
  return unexpected ? 1 : 0;
}
