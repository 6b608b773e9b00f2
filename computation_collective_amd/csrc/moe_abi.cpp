// C entry points of the mixture-of-experts operators: argument validation
// and launch-argument packing, as abi.cpp does for the fused operators.
#include <algorithm>

#include "abi_util.hpp"
#include "moe.hpp"

using namespace hocf;

namespace {

int64_t dt_bytes(hocf_dtype d) { return d == HOCF_BF16 ? 2 : 4; }

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1;

// What the router's forward and backward passes check alike.
hocf_status check_route(const char* op, int64_t T, int E, int topk, hocf_dtype dt, int64_t ld, hocf_score score,
                        int renorm, float scale) {
  if (T < 0 || T > kMaxTokens) return fail(HOCF_ERR_INVALID_ARG, "%s: T=%lld outside [0, 2^31)", op, (long long)T);
  if (E < 1 || topk < 1 || topk > E)
    return fail(HOCF_ERR_INVALID_ARG, "%s: E=%d and topk=%d must be 1 <= topk <= E", op, E, topk);
  if (!dt_ok(dt)) return fail(HOCF_ERR_INVALID_ARG, "%s: unknown dtype", op);
  if (score != HOCF_SCORE_SOFTMAX && score != HOCF_SCORE_SIGMOID)
    return fail(HOCF_ERR_INVALID_ARG, "%s: unknown score %d", op, (int)score);
  if (renorm != 0 && renorm != 1) return fail(HOCF_ERR_INVALID_ARG, "%s: renorm=%d is neither 0 nor 1", op, renorm);
  if (!(scale - scale == 0.0f)) return fail(HOCF_ERR_INVALID_ARG, "%s: scale is not finite", op);
  if (ld < E || ld > (1 << 24))
    return fail(HOCF_ERR_INVALID_ARG, "%s: ld=%lld outside [E, 2^24]", op, (long long)ld);
  if (E > kRouteMaxE || topk > kRouteMaxTopk)
    return fail(HOCF_ERR_UNSUPPORTED, "%s: E=%d > %d or topk=%d > %d", op, E, kRouteMaxE, topk, kRouteMaxTopk);
  return HOCF_OK;
}

}  // namespace

extern "C" {

/* ------------------------------------------------------------ routing */

size_t hocf_moe_route_workspace_bytes(int E) {
  return E < 1 || E > kRouteMaxE ? 0 : (size_t)(1 + kCountCopies) * route_count_stride(E) * 8;
}

hocf_status hocf_moe_route(int64_t T, int E, int topk, hocf_dtype dt, const void* logits, int64_t ld,
                           const float* bias, hocf_score score, int n_group, int topk_group, int group_top,
                           int renorm, float scale, int32_t* experts, float* weights, int32_t* counts,
                           const hocf_sync* sync, void* stream) {
  const char* op = "moe_route";
  hocf_status st = check_route(op, T, E, topk, dt, ld, score, renorm, scale);
  if (st != HOCF_OK) return st;
  if (n_group < 1 || E % n_group || topk_group < 1 || topk_group > n_group)
    return fail(HOCF_ERR_INVALID_ARG, "%s: n_group=%d must divide E=%d and hold topk_group=%d", op, n_group, E,
                topk_group);
  if (group_top != 1 && group_top != 2)
    return fail(HOCF_ERR_INVALID_ARG, "%s: group_top=%d is neither 1 nor 2", op, group_top);
  if (n_group > kRouteMaxGroups) return fail(HOCF_ERR_UNSUPPORTED, "%s: n_group=%d > %d", op, n_group, kRouteMaxGroups);
  const size_t need = counts ? hocf_moe_route_workspace_bytes(E) : 0;
  if ((st = check_sync(sync, need)) != HOCF_OK) return st;
  if (T == 0 && !counts) return ok();
  if (T && (!logits || !experts || !weights)) return fail(HOCF_ERR_INVALID_ARG, "%s: NULL tensor", op);
  if (!aligned16(logits) || !aligned16(experts) || !aligned16(weights) || !aligned16(bias) || !aligned16(counts))
    return fail(HOCF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
  {
    Ranges rg;
    if (T) rg.in("logits", 0, logits, ((T - 1) * ld + E) * dt_bytes(dt));
    rg.in("bias", 0, bias, (int64_t)E * 4);
    rg.out("experts", 0, experts, T * topk * 4);
    rg.out("weights", 0, weights, T * topk * 4);
    rg.out("counts", 0, counts, (int64_t)E * 4);
    add_sync(rg, sync, need);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  RouteArgs a{};
  a.logits = logits; a.bias = bias; a.experts = experts; a.weights = weights; a.counts = counts;
  a.ws = static_cast<uint64_t*>(sync->workspace);
  a.T = T; a.ld = ld; a.E = E; a.topk = topk; a.dt = dt; a.score = score;
  a.n_group = n_group; a.topk_group = topk_group; a.group_top = group_top;
  a.renorm = renorm; a.scale = scale;
  return launched(launch_moe_route(a, static_cast<hipStream_t>(stream)), op);
}

hocf_status hocf_moe_route_bwd(int64_t T, int E, int topk, hocf_dtype dt, const void* logits, int64_t ld,
                               const int32_t* experts, const float* dweights, hocf_score score, int renorm,
                               float scale, void* dlogits, const hocf_sync* sync, void* stream) {
  const char* op = "moe_route_bwd";
  hocf_status st = check_route(op, T, E, topk, dt, ld, score, renorm, scale);
  if (st != HOCF_OK) return st;
  if ((st = check_sync(sync, 0)) != HOCF_OK) return st;
  if (T == 0) return ok();
  if (!logits || !experts || !dweights || !dlogits) return fail(HOCF_ERR_INVALID_ARG, "%s: NULL tensor", op);
  if (!aligned16(logits) || !aligned16(experts) || !aligned16(dweights) || !aligned16(dlogits))
    return fail(HOCF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
  {
    Ranges rg;
    rg.in("logits", 0, logits, ((T - 1) * ld + E) * dt_bytes(dt));
    rg.in("experts", 0, experts, T * topk * 4);
    rg.in("dweights", 0, dweights, T * topk * 4);
    rg.out("dlogits", 0, dlogits, T * E * dt_bytes(dt));
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  RouteBwdArgs a{};
  if ((st = to_sync_args(sync, &a.sync)) != HOCF_OK) return st;
  a.logits = logits; a.experts = experts; a.dweights = dweights; a.dlogits = dlogits;
  a.T = T; a.ld = ld; a.E = E; a.topk = topk; a.dt = dt; a.score = score;
  a.renorm = renorm; a.scale = scale;
  return launched(launch_moe_route_bwd(a, static_cast<hipStream_t>(stream)), op);
}

/* ------------------------------------------------------------ window rows */

size_t hocf_moe_slots_workspace_bytes(int64_t T, int topk, int bins) {
  if (T <= 0 || topk <= 0 || bins <= 0 || T > kMaxTokens || T * topk > kMaxTokens) return 0;
  uint32_t chunk;
  int chunks;
  slots_chunks(T * topk, &chunk, &chunks);
  return (size_t)chunks * kSlotsMaxBins * 4;
}

hocf_status hocf_moe_slots(int64_t T, int topk, int bins, int per_bin, int64_t cap, const int32_t* experts,
                           int32_t* index, int32_t* pair, int64_t* counts, const hocf_sync* sync, void* stream) {
  const char* op = "moe_slots";
  if (T < 0 || T > kMaxTokens || topk < 1 || T * topk > kMaxTokens)
    return fail(HOCF_ERR_INVALID_ARG, "%s: T=%lld tokens of topk=%d outside [0, 2^31) pairs", op, (long long)T, topk);
  if (bins < 1 || per_bin < 1 || (int64_t)bins * per_bin > kMaxTokens)
    return fail(HOCF_ERR_INVALID_ARG, "%s: bins=%d of per_bin=%d experts", op, bins, per_bin);
  if (cap < 0 || cap > kMaxTokens || bins * cap > kMaxTokens)
    return fail(HOCF_ERR_INVALID_ARG, "%s: bins * cap rows outside [0, 2^31)", op);
  if (bins > kSlotsMaxBins) return fail(HOCF_ERR_UNSUPPORTED, "%s: bins=%d > %d", op, bins, kSlotsMaxBins);
  const size_t need = hocf_moe_slots_workspace_bytes(T, topk, bins);
  hocf_status st = check_sync(sync, need);
  if (st != HOCF_OK) return st;
  const int64_t pairs = T * topk;
  if (!counts || (pairs && (!experts || !index)) || (cap && !pair))
    return fail(HOCF_ERR_INVALID_ARG, "%s: NULL tensor", op);
  if (!aligned16(experts) || !aligned16(index) || !aligned16(pair) || !aligned16(counts))
    return fail(HOCF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
  {
    Ranges rg;
    rg.in("experts", 0, experts, pairs * 4);
    rg.out("index", 0, index, pairs * 4);
    rg.out("pair", 0, pair, bins * cap * 4);
    rg.out("counts", 0, counts, (int64_t)bins * 8);
    add_sync(rg, sync, need);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  SlotsArgs a{};
  a.experts = experts; a.index = index; a.pair = pair; a.counts = counts;
  a.hist = static_cast<uint32_t*>(sync->workspace);
  a.pairs = (uint32_t)pairs; a.cap = (uint32_t)cap;
  a.bins = bins; a.per_bin = per_bin; a.experts_end = (uint32_t)(bins * per_bin);
  slots_chunks(pairs, &a.chunk, &a.chunks);
  return launched(launch_moe_slots(a, static_cast<hipStream_t>(stream)), op);
}

/* ------------------------------------------------------------ weighted sum */

// What the combine's forward and backward passes check alike.
static hocf_status check_combine(const char* op, int64_t T, int topk, int N, int64_t R, hocf_dtype dt,
                                 hocf_dtype out_dt, const void* index, const hocf_sync* sync) {
  if (T < 0 || T > kMaxTokens || R < 0 || R > kMaxTokens || topk < 1 || N < 0)
    return fail(HOCF_ERR_INVALID_ARG, "%s: T=%lld R=%lld topk=%d N=%d out of range", op, (long long)T, (long long)R,
                topk, N);
  if (!dt_ok(dt) || !dt_ok(out_dt)) return fail(HOCF_ERR_INVALID_ARG, "%s: unknown dtype", op);
  if (N % 8) return fail(HOCF_ERR_INVALID_ARG, "%s: N=%d not a multiple of 8", op, N);
  if (!index && T && R != T * topk)
    return fail(HOCF_ERR_INVALID_ARG, "%s: without an index R=%lld must be T * topk", op, (long long)R);
  if (topk > kRouteMaxTopk || N > (1 << 24))
    return fail(HOCF_ERR_UNSUPPORTED, "%s: topk=%d > %d or N=%d > 2^24", op, topk, kRouteMaxTopk, N);
  return check_sync(sync, 0);
}

hocf_status hocf_moe_combine(int64_t T, int topk, int N, int64_t R, hocf_dtype dt, hocf_dtype out_dt,
                             const void* rows, const float* weights, const int32_t* index, const void* add,
                             void* out, const hocf_sync* sync, void* stream) {
  const char* op = "moe_combine";
  hocf_status st = check_combine(op, T, topk, N, R, dt, out_dt, index, sync);
  if (st != HOCF_OK) return st;
  if (T == 0 || N == 0) return ok();
  if ((R && !rows) || !weights || !out) return fail(HOCF_ERR_INVALID_ARG, "%s: NULL tensor", op);
  if (!aligned16(rows) || !aligned16(weights) || !aligned16(index) || !aligned16(add) || !aligned16(out))
    return fail(HOCF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
  {
    Ranges rg;
    rg.in("rows", 0, rows, R * N * dt_bytes(dt));
    rg.in("weights", 0, weights, T * topk * 4);
    rg.in("index", 0, index, T * topk * 4);
    rg.in("add", 0, add, T * N * dt_bytes(out_dt));
    rg.out("out", 0, out, T * N * dt_bytes(out_dt));
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  CombineArgs a{};
  if ((st = to_sync_args(sync, &a.sync)) != HOCF_OK) return st;
  a.rows = rows; a.weights = weights; a.index = index; a.add = add; a.out = out;
  a.T = T; a.R = R; a.topk = topk; a.N = N; a.dt = dt; a.out_dt = out_dt;
  return launched(launch_moe_combine(a, static_cast<hipStream_t>(stream)), op);
}

hocf_status hocf_moe_combine_bwd(int64_t T, int topk, int N, int64_t R, hocf_dtype dt, hocf_dtype out_dt,
                                 const void* rows, const float* weights, const void* dout, const int32_t* index,
                                 const int32_t* pair, void* drows, float* dweights, const hocf_sync* sync,
                                 void* stream) {
  const char* op = "moe_combine_bwd";
  hocf_status st = check_combine(op, T, topk, N, R, dt, out_dt, index, sync);
  if (st != HOCF_OK) return st;
  if (T ? (R && !index != !pair) : (R && !pair))
    return fail(HOCF_ERR_INVALID_ARG, "%s: index and pair go together", op);
  if (T == 0 && R == 0) return ok();
  if ((T && (!weights || !dweights)) || (N && ((T && !dout) || (R && (!rows || !drows)))))
    return fail(HOCF_ERR_INVALID_ARG, "%s: NULL tensor", op);
  if (!aligned16(rows) || !aligned16(weights) || !aligned16(dout) || !aligned16(index) || !aligned16(pair) ||
      !aligned16(drows) || !aligned16(dweights))
    return fail(HOCF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
  {
    Ranges rg;
    rg.in("rows", 0, rows, R * N * dt_bytes(dt));
    rg.in("weights", 0, weights, T * topk * 4);
    rg.in("dout", 0, dout, T * N * dt_bytes(out_dt));
    rg.in("index", 0, index, T * topk * 4);
    rg.in("pair", 0, pair, R * 4);
    rg.out("drows", 0, drows, R * N * dt_bytes(dt));
    rg.out("dweights", 0, dweights, T * topk * 4);
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  CombineArgs a{};
  if ((st = to_sync_args(sync, &a.sync)) != HOCF_OK) return st;
  a.rows = rows; a.weights = weights; a.dout = dout; a.index = index; a.pair = pair;
  a.drows = drows; a.dweights = dweights;
  a.T = T; a.R = R; a.topk = topk; a.N = N; a.dt = dt; a.out_dt = out_dt;
  return launched(launch_moe_combine_bwd(a, static_cast<hipStream_t>(stream)), op);
}

/* ------------------------------------------------------------ 4-bit weights */

// What the product and the packing check alike.
static hocf_status check_w4(const char* op, int E, int N, int K, int group) {
  if (E < 1 || N < 0 || K < 0 || N % 8 || K % 8)
    return fail(HOCF_ERR_INVALID_ARG, "%s: E=%d, N=%d and K=%d: E >= 1, N and K multiples of 8", op, E, N, K);
  if (group != 32 && group != 64 && group != 128)
    return fail(HOCF_ERR_UNSUPPORTED, "%s: group=%d is none of 32, 64, 128", op, group);
  if (N > (1 << 20) || K > (1 << 20)) return fail(HOCF_ERR_UNSUPPORTED, "%s: N=%d or K=%d > 2^20", op, N, K);
  // (no memory holds these; their sizes in bytes would not fit 64 bits)
  if (E > (int64_t(1) << 60) / std::max<int64_t>(cdiv(N, 16) * 16 * cdiv(K, 128) * 128, 1))
    return fail(HOCF_ERR_UNSUPPORTED, "%s: E=%d experts of %d x %d are more than 2^60 weights", op, E, K, N);
  return HOCF_OK;
}

hocf_status hocf_gemv_w4(int R, int rows_per_x, int E, int e0, int N, int K, int group, hocf_dtype out_dt,
                         const void* x, const int32_t* experts, const uint32_t* wq, const void* scales,
                         const void* zeros, void* out, const hocf_sync* sync, void* stream) {
  const char* op = "gemv_w4";
  hocf_status st = check_w4(op, E, N, K, group);
  if (st != HOCF_OK) return st;
  if (R < 0 || rows_per_x < 1 || R % rows_per_x)
    return fail(HOCF_ERR_INVALID_ARG, "%s: R=%d must be a multiple of rows_per_x=%d", op, R, rows_per_x);
  if (!dt_ok(out_dt)) return fail(HOCF_ERR_INVALID_ARG, "%s: unknown dtype", op);
  if (e0 < 0 || e0 > kMaxTokens - E) return fail(HOCF_ERR_INVALID_ARG, "%s: e0=%d with E=%d experts", op, e0, E);
  if (!experts && E != 1) return fail(HOCF_ERR_INVALID_ARG, "%s: E=%d experts need the rows' choices", op, E);
  if (R > kW4MaxRows) return fail(HOCF_ERR_UNSUPPORTED, "%s: R=%d > %d rows", op, R, kW4MaxRows);
  if ((st = check_sync(sync, 0)) != HOCF_OK) return st;
  if (R == 0 || N == 0) return ok();
  if (!out || (K && (!x || !wq || !scales))) return fail(HOCF_ERR_INVALID_ARG, "%s: NULL tensor", op);
  if (!aligned16(x) || !aligned16(experts) || !aligned16(wq) || !aligned16(scales) || !aligned16(zeros) ||
      !aligned16(out))
    return fail(HOCF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
  GemvW4Args a{};
  a.nb = (int)cdiv(N, 16);
  a.kb = (int)cdiv(K, 128);
  a.groups = (int)cdiv(K, group);
  {
    const int64_t sc = (int64_t)E * a.nb * a.groups * 32;
    Ranges rg;
    rg.in("x", 0, x, (int64_t)(R / rows_per_x) * K * 2);
    rg.in("experts", 0, experts, (int64_t)R * 4);
    rg.in("wq", 0, wq, (int64_t)E * a.nb * a.kb * 1024);
    rg.in("scales", 0, scales, sc);
    rg.in("zeros", 0, zeros, sc);
    rg.out("out", 0, out, (int64_t)R * N * dt_bytes(out_dt));
    add_sync(rg, sync, 0);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  a.x = static_cast<const uint16_t*>(x);
  a.experts = experts; a.wq = wq;
  a.scales = static_cast<const uint16_t*>(scales);
  a.zeros = static_cast<const uint16_t*>(zeros);
  a.out = out;
  a.R = R; a.rows_per_x = rows_per_x; a.E = E; a.e0 = e0; a.N = N; a.K = K; a.group = group; a.out_dt = out_dt;
  return launched(launch_gemv_w4(a, static_cast<hipStream_t>(stream)), op);
}

hocf_status hocf_w4_pack(int E, int N, int K, int group, const uint8_t* codes, const void* scales, const void* zeros,
                         uint32_t* wq, void* scales_out, void* zeros_out, void* stream) {
  const char* op = "w4_pack";
  hocf_status st = check_w4(op, E, N, K, group);
  if (st != HOCF_OK) return st;
  if (!zeros != !zeros_out) return fail(HOCF_ERR_INVALID_ARG, "%s: zeros and zeros_out go together", op);
  if (N == 0 || K == 0) return ok();
  if (!codes || !scales || !wq || !scales_out) return fail(HOCF_ERR_INVALID_ARG, "%s: NULL tensor", op);
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(zeros) || !aligned16(wq) || !aligned16(scales_out) ||
      !aligned16(zeros_out))
    return fail(HOCF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
  W4PackArgs a{};
  a.E = E; a.N = N; a.K = K;
  a.nb = (int)cdiv(N, 16);
  a.kb = (int)cdiv(K, 128);
  a.groups = (int)cdiv(K, group);
  {
    const int64_t in = (int64_t)E * a.groups * N * 2, sc = (int64_t)E * a.nb * a.groups * 32;
    Ranges rg;
    rg.in("codes", 0, codes, (int64_t)E * K * N);
    rg.in("scales", 0, scales, in);
    rg.in("zeros", 0, zeros, in);
    rg.out("wq", 0, wq, (int64_t)E * a.nb * a.kb * 1024);
    rg.out("scales_out", 0, scales_out, sc);
    rg.out("zeros_out", 0, zeros_out, sc);
    if ((st = rg.check(op)) != HOCF_OK) return st;
  }
  a.codes = codes;
  a.scales = static_cast<const uint16_t*>(scales);
  a.zeros = static_cast<const uint16_t*>(zeros);
  a.wq = wq;
  a.scales_out = static_cast<uint16_t*>(scales_out);
  a.zeros_out = static_cast<uint16_t*>(zeros_out);
  return launched(launch_w4_pack(a, static_cast<hipStream_t>(stream)), op);
}

}  // extern "C"
