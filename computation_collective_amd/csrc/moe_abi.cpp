// C entry points of the mixture-of-experts operators: argument validation
// and launch-argument packing, as abi.cpp does for the fused operators.
#include "abi_util.hpp"
#include "moe.hpp"

using namespace hocf;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

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

size_t hocf_moe_route_workspace_bytes(int E) { return E < 1 ? 0 : (size_t)(1 + E) * 4; }

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
  a.ws = static_cast<uint32_t*>(sync->workspace);
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

}  // extern "C"
