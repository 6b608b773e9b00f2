// Launch-side declarations of the mixture-of-experts operators (moe_abi.cpp
// checks the arguments, the moe_*.hip and gemv_w4.hip units launch).
#pragma once

#include "internal.hpp"

namespace hocf {

constexpr int kRouteMaxE = 512;     // experts of one router row
constexpr int kRouteMaxTopk = 16;   // choices of one token
constexpr int kRouteMaxGroups = 64;

enum Score : int { kSoftmax = 0, kSigmoid = 1 };

struct RouteArgs {
  const void* logits;  // [T][ld] dt
  const float* bias;   // [E] or NULL
  int32_t* experts;    // [T][topk]
  float* weights;      // [T][topk]
  int32_t* counts;     // [E] or NULL
  uint32_t* ws;        // with counts: [0] workgroups that have finished, [1 .. 1 + E) their counts; all left zeroed
  int64_t T, ld;
  int E, topk, dt, score, n_group, topk_group, group_top, renorm;
  float scale;
};

struct RouteBwdArgs {
  const void* logits;       // [T][ld] dt
  const int32_t* experts;   // [T][topk]
  const float* dweights;    // [T][topk]
  void* dlogits;            // [T][E] dt
  int64_t T, ld;
  int E, topk, dt, score, renorm;
  float scale;
  SyncArgs sync;
};

int launch_moe_route(const RouteArgs& a, hipStream_t s);
int launch_moe_route_bwd(const RouteBwdArgs& a, hipStream_t s);

}  // namespace hocf
