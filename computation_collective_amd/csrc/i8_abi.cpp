// C entry points of the 8-bit integer operators: argument validation and
// launch-argument packing, as abi.cpp does for the fused operators.
#include "abi_util.hpp"
#include "i8.hpp"

using namespace hocf;

namespace {

int64_t dt_bytes(hocf_dtype d) { return d == HOCF_BF16 ? 2 : 4; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

hocf_status check_rows(const char* op, int64_t T) {
  if (T < 0 || T > kMaxRows) return fail(HOCF_ERR_INVALID_ARG, "%s: T=%lld outside [0, 2^31)", op, (long long)T);
  return HOCF_OK;
}
hocf_status check_k(const char* op, int K) {
  if (K < 16 || K % 16) return fail(HOCF_ERR_INVALID_ARG, "%s: K=%d is no positive multiple of 16", op, K);
  if (K > kI8MaxDim) return fail(HOCF_ERR_UNSUPPORTED, "%s: K=%d > %d", op, K, kI8MaxDim);
  return HOCF_OK;
}
// The sizes of E matrices of codes.
hocf_status check_matrices(const char* op, int E, int N, int K) {
  if (E < 1) return fail(HOCF_ERR_INVALID_ARG, "%s: E=%d < 1", op, E);
  if (N < 8 || N % 8) return fail(HOCF_ERR_INVALID_ARG, "%s: N=%d is no positive multiple of 8", op, N);
  const hocf_status st = check_k(op, K);
  if (st != HOCF_OK) return st;
  if (E > kI8MaxExperts || N > kI8MaxDim)
    return fail(HOCF_ERR_UNSUPPORTED, "%s: E=%d > %d or N=%d > %d", op, E, kI8MaxExperts, N, kI8MaxDim);
  return HOCF_OK;
}
hocf_status check_grouped(const char* op, int E, int64_t T, int N, int K, hocf_dtype out_dt, const int64_t* offsets,
                          const hocf_sync* sync) {
  hocf_status st = check_matrices(op, E, N, K);
  if (st != HOCF_OK || (st = check_rows(op, T)) != HOCF_OK) return st;
  if (!dt_ok(out_dt)) return fail(HOCF_ERR_INVALID_ARG, "%s: unknown dtype", op);
  if (!offsets && E != 1) return fail(HOCF_ERR_INVALID_ARG, "%s: E=%d experts need their groups' offsets", op, E);
  return check_sync(sync, 0);
}
template <class... P>
hocf_status check_aligned(const char* op, P... p) {
  const bool all = (aligned16(p) && ...);
  return all ? HOCF_OK : fail(HOCF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
}
hocf_status null_tensor(const char* op) { return fail(HOCF_ERR_INVALID_ARG, "%s: NULL tensor", op); }

}  // namespace

extern "C" {

/* ------------------------------------------------------------ rows */

hocf_status hocf_quant_i8(int64_t T, int K, hocf_dtype dt, const void* x, int64_t ld, hocf_act act, int8_t* codes,
                          float* scales, int8_t* pre_codes, float* pre_scales, const hocf_sync* sync, void* stream) {
  const char* op = "quant_i8";
  hocf_status st = check_rows(op, T);
  if (st != HOCF_OK || (st = check_k(op, K)) != HOCF_OK) return st;
  if (!dt_ok(dt)) return fail(HOCF_ERR_INVALID_ARG, "%s: unknown dtype", op);
  if (act != HOCF_ACT_NONE && act != HOCF_ACT_SILU)
    return fail(HOCF_ERR_INVALID_ARG, "%s: unknown activation %d", op, (int)act);
  if (ld < K || ld > (1 << 24) || ld * dt_bytes(dt) % 16)
    return fail(HOCF_ERR_INVALID_ARG, "%s: ld=%lld outside [K, 2^24], or rows not 16-byte aligned", op, (long long)ld);
  if (!pre_codes != !pre_scales)
    return fail(HOCF_ERR_INVALID_ARG, "%s: pre_codes and pre_scales go together", op);
  if (pre_codes && act == HOCF_ACT_NONE)
    return fail(HOCF_ERR_INVALID_ARG, "%s: without an activation the codes are those of x already", op);
  if ((st = check_sync(sync, 0)) != HOCF_OK) return st;
  if (T == 0) return ok();
  if (!x || !codes || !scales) return null_tensor(op);
  if ((st = check_aligned(op, x, codes, scales, pre_codes, pre_scales)) != HOCF_OK) return st;
  {
    Ranges rg;
    rg.in("x", 0, x, ((T - 1) * ld + K) * dt_bytes(dt));
    rg.out("codes", 0, codes, T * K);
    rg.out("scales", 0, scales, T * 4);
    rg.out("pre_codes", 0, pre_codes, T * K);
    rg.out("pre_scales", 0, pre_scales, T * 4);
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  QuantI8Args a{};
  a.x = x; a.codes = codes; a.scales = scales; a.pre_codes = pre_codes; a.pre_scales = pre_scales;
  a.T = T; a.ld = ld; a.K = K; a.dt = dt; a.act = act;
  return launched(launch_quant_i8(a, static_cast<hipStream_t>(stream)), op);
}

hocf_status hocf_dequant_i8(int64_t T, int K, hocf_dtype out_dt, const int8_t* codes, const float* scales, void* out,
                            const hocf_sync* sync, void* stream) {
  const char* op = "dequant_i8";
  hocf_status st = check_rows(op, T);
  if (st != HOCF_OK || (st = check_k(op, K)) != HOCF_OK) return st;
  if (!dt_ok(out_dt)) return fail(HOCF_ERR_INVALID_ARG, "%s: unknown dtype", op);
  if ((st = check_sync(sync, 0)) != HOCF_OK) return st;
  if (T == 0) return ok();
  if (!codes || !scales || !out) return null_tensor(op);
  if ((st = check_aligned(op, codes, scales, out)) != HOCF_OK) return st;
  {
    Ranges rg;
    rg.in("codes", 0, codes, T * K);
    rg.in("scales", 0, scales, T * 4);
    rg.out("out", 0, out, T * K * dt_bytes(out_dt));
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  DequantI8Args a{};
  a.codes = codes; a.scales = scales; a.out = out; a.T = T; a.K = K; a.dt = out_dt;
  return launched(launch_dequant_i8(a, static_cast<hipStream_t>(stream)), op);
}

/* ------------------------------------------------------------ weights */

size_t hocf_weights_i8_workspace_bytes(int E, int N, int K) {
  if (E < 1 || N < 1 || K < 1 || E > kI8MaxExperts || N > kI8MaxDim || K > kI8MaxDim) return 0;
  return (size_t)E * w8_slabs(K) * N * 4;
}

hocf_status hocf_weights_i8(int E, int N, int K, hocf_dtype dt, const void* W, int8_t* wq, float* scales,
                            const hocf_sync* sync, void* stream) {
  const char* op = "weights_i8";
  hocf_status st = check_matrices(op, E, N, K);
  if (st != HOCF_OK) return st;
  if (!dt_ok(dt)) return fail(HOCF_ERR_INVALID_ARG, "%s: unknown dtype", op);
  const size_t need = hocf_weights_i8_workspace_bytes(E, N, K);
  if ((st = check_sync(sync, need)) != HOCF_OK) return st;
  if (!W || !wq || !scales) return null_tensor(op);
  if ((st = check_aligned(op, W, wq, scales)) != HOCF_OK) return st;
  {
    Ranges rg;
    rg.in("W", 0, W, (int64_t)E * K * N * dt_bytes(dt));
    rg.out("wq", 0, wq, (int64_t)E * N * K);
    rg.out("scales", 0, scales, (int64_t)E * N * 4);
    add_sync(rg, sync, need);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  WeightsI8Args a{};
  a.W = W; a.wq = wq; a.scales = scales; a.part = static_cast<uint32_t*>(sync->workspace);
  a.E = E; a.N = N; a.K = K; a.dt = dt; a.slabs = w8_slabs(K);
  return launched(launch_weights_i8(a, static_cast<hipStream_t>(stream)), op);
}

/* ------------------------------------------------------------ products */

hocf_status hocf_gemm_i8(int E, int64_t T, int N, int K, hocf_dtype out_dt, const int8_t* xq, const float* xs,
                         const int8_t* wq, const float* ws, const int64_t* offsets, void* out, const hocf_sync* sync,
                         void* stream) {
  const char* op = "gemm_i8";
  hocf_status st = check_grouped(op, E, T, N, K, out_dt, offsets, sync);
  if (st != HOCF_OK) return st;
  if (T == 0) return ok();
  if (!xq || !xs || !wq || !ws || !out) return null_tensor(op);
  if ((st = check_aligned(op, xq, xs, wq, ws, offsets, out)) != HOCF_OK) return st;
  {
    Ranges rg;
    rg.in("xq", 0, xq, T * K);
    rg.in("xs", 0, xs, T * 4);
    rg.in("wq", 0, wq, (int64_t)E * N * K);
    rg.in("ws", 0, ws, (int64_t)E * N * 4);
    rg.in("offsets", 0, offsets, (int64_t)(E + 1) * 8);
    rg.out("out", 0, out, T * N * dt_bytes(out_dt));
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  GemmI8Args a{};
  if ((st = to_sync_args(sync, &a.sync)) != HOCF_OK) return st;
  a.xq = xq; a.xs = xs; a.wq = wq; a.ws = ws; a.offsets = offsets; a.out = out;
  a.T = T; a.E = E; a.N = N; a.K = K; a.out_dt = out_dt;
  return launched(launch_gemm_i8(a, static_cast<hipStream_t>(stream)), op);
}

hocf_status hocf_gemv_i8(int R, int rows_per_x, int E, int e0, int N, int K, hocf_dtype out_dt, const int8_t* xq,
                         const float* xs, const int32_t* experts, const int8_t* wq, const float* ws, void* out,
                         const hocf_sync* sync, void* stream) {
  const char* op = "gemv_i8";
  hocf_status st = check_matrices(op, E, N, K);
  if (st != HOCF_OK) return st;
  if (R < 0 || rows_per_x < 1 || R % rows_per_x)
    return fail(HOCF_ERR_INVALID_ARG, "%s: R=%d must be a multiple of rows_per_x=%d", op, R, rows_per_x);
  if (!dt_ok(out_dt)) return fail(HOCF_ERR_INVALID_ARG, "%s: unknown dtype", op);
  if (e0 < 0 || e0 > kMaxRows - E) return fail(HOCF_ERR_INVALID_ARG, "%s: e0=%d with E=%d experts", op, e0, E);
  if (!experts && E != 1) return fail(HOCF_ERR_INVALID_ARG, "%s: E=%d experts need the rows' choices", op, E);
  if (R > kI8MaxRows) return fail(HOCF_ERR_UNSUPPORTED, "%s: R=%d > %d rows", op, R, kI8MaxRows);
  if ((st = check_sync(sync, 0)) != HOCF_OK) return st;
  if (R == 0) return ok();
  if (!xq || !xs || !wq || !ws || !out) return null_tensor(op);
  if ((st = check_aligned(op, xq, xs, experts, wq, ws, out)) != HOCF_OK) return st;
  {
    Ranges rg;
    rg.in("xq", 0, xq, (int64_t)(R / rows_per_x) * K);
    rg.in("xs", 0, xs, (int64_t)(R / rows_per_x) * 4);
    rg.in("experts", 0, experts, (int64_t)R * 4);
    rg.in("wq", 0, wq, (int64_t)E * N * K);
    rg.in("ws", 0, ws, (int64_t)E * N * 4);
    rg.out("out", 0, out, (int64_t)R * N * dt_bytes(out_dt));
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  GemvI8Args a{};
  a.xq = xq; a.xs = xs; a.experts = experts; a.wq = wq; a.ws = ws; a.out = out;
  a.R = R; a.rows_per_x = rows_per_x; a.E = E; a.e0 = e0; a.N = N; a.K = K; a.out_dt = out_dt;
  return launched(launch_gemv_i8(a, static_cast<hipStream_t>(stream)), op);
}

/* ------------------------------------------------------------ gradients */

hocf_status hocf_gemm_i8_dx(int E, int64_t T, int N, int K, hocf_dtype out_dt, const void* dy, const int8_t* wq,
                            const float* ws, const int64_t* offsets, const int8_t* pre_codes, const float* pre_scales,
                            void* dx, const hocf_sync* sync, void* stream) {
  const char* op = "gemm_i8_dx";
  hocf_status st = check_grouped(op, E, T, N, K, out_dt, offsets, sync);
  if (st != HOCF_OK) return st;
  if (!pre_codes != !pre_scales)
    return fail(HOCF_ERR_INVALID_ARG, "%s: pre_codes and pre_scales go together", op);
  if (T == 0) return ok();
  if (!dy || !wq || !ws || !dx) return null_tensor(op);
  if ((st = check_aligned(op, dy, wq, ws, offsets, pre_codes, pre_scales, dx)) != HOCF_OK) return st;
  {
    Ranges rg;
    rg.in("dy", 0, dy, T * N * 2);
    rg.in("wq", 0, wq, (int64_t)E * N * K);
    rg.in("ws", 0, ws, (int64_t)E * N * 4);
    rg.in("offsets", 0, offsets, (int64_t)(E + 1) * 8);
    rg.in("pre_codes", 0, pre_codes, T * K);
    rg.in("pre_scales", 0, pre_scales, T * 4);
    rg.out("dx", 0, dx, T * K * dt_bytes(out_dt));
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  GradI8Args a{};
  if ((st = to_sync_args(sync, &a.sync)) != HOCF_OK) return st;
  a.dy = static_cast<const uint16_t*>(dy);
  a.q = wq; a.s = ws; a.offsets = offsets; a.pre = pre_codes; a.pre_s = pre_scales; a.out = dx;
  a.T = T; a.E = E; a.N = N; a.K = K; a.out_dt = out_dt;
  return launched(launch_gemm_i8_dx(a, static_cast<hipStream_t>(stream)), op);
}

size_t hocf_gemm_i8_dw_workspace_bytes(int E, int64_t T, int N, int K) {
  if (E < 1 || T < 1 || N < 1 || K < 1 || E > kI8MaxExperts || T > kMaxRows || N > kI8MaxDim || K > kI8MaxDim) return 0;
  const int splits = dw_splits(E, T, N, K);
  return splits > 1 ? (size_t)splits * E * K * N * 4 : 0;
}

hocf_status hocf_gemm_i8_dw(int E, int64_t T, int N, int K, hocf_dtype out_dt, const int8_t* xq, const float* xs,
                            const void* dy, const int64_t* offsets, void* dw, const hocf_sync* sync, void* stream) {
  const char* op = "gemm_i8_dw";
  hocf_status st = check_grouped(op, E, T, N, K, out_dt, offsets, sync);
  if (st != HOCF_OK) return st;
  const size_t need = hocf_gemm_i8_dw_workspace_bytes(E, T, N, K);
  if ((st = check_sync(sync, need)) != HOCF_OK) return st;
  if ((T && (!xq || !xs || !dy)) || !dw) return null_tensor(op);
  if ((st = check_aligned(op, xq, xs, dy, offsets, dw)) != HOCF_OK) return st;
  {
    Ranges rg;
    rg.in("xq", 0, xq, T * K);
    rg.in("xs", 0, xs, T * 4);
    rg.in("dy", 0, dy, T * N * 2);
    rg.in("offsets", 0, offsets, (int64_t)(E + 1) * 8);
    rg.out("dw", 0, dw, (int64_t)E * K * N * dt_bytes(out_dt));
    add_sync(rg, sync, need);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  GradI8Args a{};
  if ((st = to_sync_args(sync, &a.sync)) != HOCF_OK) return st;
  a.dy = static_cast<const uint16_t*>(dy);
  a.q = xq; a.s = xs; a.offsets = offsets; a.out = dw;
  a.part = static_cast<float*>(sync->workspace);
  a.T = T; a.E = E; a.N = N; a.K = K; a.out_dt = out_dt;
  return launched(launch_gemm_i8_dw(a, static_cast<hipStream_t>(stream)), op);
}

}  // extern "C"
