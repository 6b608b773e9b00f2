// The argument validation of the 8-bit integer entries, built with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host code by
// tests/test_sanitize_i8_cpu.py: every integer argument at the ends of its
// type and around its limits, alone and against one other argument's.  Every
// call is to fail: the sync block is invalid (the arithmetic of the checks
// before it), or all tensors are one (the sizes of the ranges).  The pointers
// are fake addresses, never dereferenced.  Exit status 0 when every call
// returned an error, or HOCF_OK for a call with nothing to do.
#include <climits>
#include <cstdint>
#include <cstdio>

#include "hocf.h"

static const int64_t kEnds[] = {INT64_MIN, INT64_MAX, INT_MIN, INT_MAX, -1, 0, 1, 2, 7, 8, 16, 17, 128, 1024, 1025, 65536, 65544,
                                65552, 1 << 20, 1 << 24, int64_t(1) << 31, (int64_t(1) << 31) - 8, int64_t(1) << 40};
static long calls = 0, unexpected = 0;

// Calls fn on the base arguments with every end in every place, and in every pair of places.
template <int N, class FN>
static void sweep(const char* name, const int64_t (&base)[N], FN fn) {
  for (int i = 0; i < N; ++i)
    for (int64_t u : kEnds)
      for (int j = i; j < N; ++j)
        for (int64_t v : kEnds) {
          int64_t a[N];
          for (int k = 0; k < N; ++k) a[k] = base[k];
          a[i] = u;
          if (j > i) a[j] = v;
          const hocf_status st = fn(a);
          ++calls;
          if ((st == HOCF_ERR_HIP || (int)st < 0 || (int)st > HOCF_ERR_CAPACITY) && ++unexpected <= 10)
            std::fprintf(stderr, "%s: status %d (%s)\n", name, (int)st, hocf_last_error());
          if (j == i) break;
        }
}

int main() {
  char* const p = reinterpret_cast<char*>(uintptr_t(1) << 44);
  int8_t* const i8 = reinterpret_cast<int8_t*>(p);
  int32_t* const i32 = reinterpret_cast<int32_t*>(p);
  int64_t* const i64 = reinterpret_cast<int64_t*>(p);
  float* const f = reinterpret_cast<float*>(p);
  hocf_sync one{};  // (its workspace is the tensors' memory too)
  one.epoch = 1;
  one.workspace = p;
  one.workspace_bytes = size_t(1) << 50;
  one.status = reinterpret_cast<uint32_t*>(p);
  hocf_sync bad = one;
  bad.epoch = 0;
  const hocf_sync* syncs[] = {&bad, &one};
  auto dt = [](int64_t v) { return static_cast<hocf_dtype>((int)v); };

  for (const hocf_sync* s : syncs) {
    for (int8_t* pre : {i8, (int8_t*)nullptr}) {
      sweep("quant_i8", {100, 64, HOCF_BF16, 64, HOCF_ACT_SILU}, [&](const int64_t(&a)[5]) {
        return hocf_quant_i8(a[0], (int)a[1], dt(a[2]), p, a[3], static_cast<hocf_act>((int)a[4]), i8, f, pre,
                             pre ? f : nullptr, s, nullptr);
      });
      sweep("gemm_i8_dx", {4, 100, 64, 128, HOCF_F32}, [&](const int64_t(&a)[5]) {
        return hocf_gemm_i8_dx((int)a[0], a[1], (int)a[2], (int)a[3], dt(a[4]), p, i8, f, i64, pre, pre ? f : nullptr, p, s,
                               nullptr);
      });
    }
    sweep("dequant_i8", {100, 64, HOCF_F32}, [&](const int64_t(&a)[3]) {
      return hocf_dequant_i8(a[0], (int)a[1], dt(a[2]), i8, f, p, s, nullptr);
    });
    sweep("weights_i8", {4, 64, 128, HOCF_F32}, [&](const int64_t(&a)[4]) {
      return hocf_weights_i8((int)a[0], (int)a[1], (int)a[2], dt(a[3]), p, i8, f, s, nullptr);
    });
    for (int64_t* off : {i64, (int64_t*)nullptr}) {
      sweep("gemm_i8", {off ? 4 : 1, 100, 64, 128, HOCF_BF16}, [&](const int64_t(&a)[5]) {
        return hocf_gemm_i8((int)a[0], a[1], (int)a[2], (int)a[3], dt(a[4]), i8, f, i8, f, off, p, s, nullptr);
      });
      sweep("gemm_i8_dw", {off ? 4 : 1, 100, 64, 128, HOCF_F32}, [&](const int64_t(&a)[5]) {
        return hocf_gemm_i8_dw((int)a[0], a[1], (int)a[2], (int)a[3], dt(a[4]), i8, f, p, off, p, s, nullptr);
      });
    }
    sweep("gemv_i8", {8, 2, 4, 0, 64, 128, HOCF_F32}, [&](const int64_t(&a)[7]) {
      return hocf_gemv_i8((int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)a[4], (int)a[5], dt(a[6]), i8, f, i32, i8, f, p, s,
                          nullptr);
    });
  }
  for (int64_t a : kEnds)
    for (int64_t b : kEnds)
      for (int64_t c : kEnds) (void)hocf_weights_i8_workspace_bytes((int)a, (int)b, (int)c);
  std::printf("i8 abi driver: %ld calls, %ld failures\n", calls, unexpected);
  return unexpected ? 1 : 0;
}
