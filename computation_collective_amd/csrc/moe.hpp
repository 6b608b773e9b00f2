// Launch-side declarations of the mixture-of-experts operators (moe_abi.cpp
// checks the arguments, the moe_*.hip and gemv_w4.hip units launch).
#pragma once

#include <algorithm>

#include "internal.hpp"

namespace hocf {

constexpr int kRouteMaxE = 512;     // experts of one router row
constexpr int kRouteMaxTopk = 16;   // choices of one token
constexpr int kRouteMaxGroups = 64;

// With counts, the router's workspace: a table of the experts' counts, then
// kCountCopies tables that workgroups add to, 64 bits a word; all left zeroed.
constexpr int kCountCopies = 8;
__host__ __device__ constexpr int route_count_stride(int E) { return (E + 15) / 16 * 16; }

enum Score : int { kSoftmax = 0, kSigmoid = 1 };

struct RouteArgs {
  const void* logits;  // [T][ld] dt
  const float* bias;   // [E] or NULL
  int32_t* experts;    // [T][topk]
  float* weights;      // [T][topk]
  int32_t* counts;     // [E] or NULL
  uint64_t* ws;        // with counts
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

constexpr int kSlotsMaxBins = 64;   // one lane counts one bin
constexpr int kSlotsThreads = 1024;
constexpr int kSlotsMaxChunks = 256;

struct SlotsArgs {
  const int32_t* experts;  // [pairs]
  int32_t* index;          // [pairs]
  int32_t* pair;           // [bins * cap]
  int64_t* counts;         // [bins]
  uint32_t* hist;          // workspace (chunked form only): the chunks' pairs of each bin
  uint32_t pairs, chunk;   // chunk: pairs of one workgroup, a multiple of kSlotsThreads
  uint32_t cap, experts_end;  // experts_end = bins * per_bin
  int bins, per_bin, chunks;
};

struct CombineArgs {
  const void* rows;      // [R][N] dt
  const float* weights;  // [T][topk]
  const int32_t* index;  // [T][topk] or NULL
  const int32_t* pair;   // [R] or NULL (backward)
  const void* add;       // [T][N] out_dt or NULL (forward)
  const void* dout;      // [T][N] out_dt (backward)
  void* out;             // [T][N] out_dt (forward)
  void* drows;           // [R][N] dt (backward)
  float* dweights;       // [T][topk] (backward)
  int64_t T, R;
  int topk, N, dt, out_dt;
  SyncArgs sync;
};

// How the weighted sum's backward pass gives a call's tokens to waves.
enum BwdForm { kWide, kRows, kShifted };

// Four waves on a token where tokens alone would not fill the device, and where
// the rows hold nothing (the shifted form reads a piece of every row it is given).
// Else a wave each, on pieces that start where the rows' cache lines do.
constexpr int kLine = 128;  // bytes of a cache line
constexpr BwdForm combine_bwd_form(int64_t T, int64_t R, int N, int dt, uintptr_t drows) {
  if (T < 2048 || R == 0 || N == 0) return kWide;
  return (int64_t)N * (dt == kBF16 ? 2 : 4) % kLine == 0 && drows % kLine == 0 ? kRows : kShifted;
}

constexpr int kW4MaxRows = 1024;

struct GemvW4Args {
  const uint16_t* x;       // [R / rows_per_x][K]
  const int32_t* experts;  // [R] or NULL
  const uint32_t* wq;      // [E][nb][kb][64][4]
  const uint16_t* scales;  // [E][nb][groups][16]
  const uint16_t* zeros;   // the same, or NULL
  void* out;               // [R][N] out_dt
  int R, rows_per_x, E, e0, N, K, group, out_dt;
  int nb, kb, groups;      // ceil(N / 16), ceil(K / 128), ceil(K / group)
};

struct W4PackArgs {
  const uint8_t* codes;    // [E][K][N]
  const uint16_t *scales, *zeros;  // [E][groups][N]
  uint32_t* wq;
  uint16_t *scales_out, *zeros_out;
  int E, N, K, nb, kb, groups;
};

int launch_gemv_w4(const GemvW4Args& a, hipStream_t s);
int launch_w4_pack(const W4PackArgs& a, hipStream_t s);

// Pairs of one chunk, and how many chunks, for a number of pairs: a chunk for
// every CU, and at most kSlotsMaxChunks.
inline void slots_chunks(int64_t pairs, uint32_t* chunk, int* chunks) {
  const int64_t c = (pairs + (int64_t)kSlotsMaxChunks * kSlotsThreads - 1) / ((int64_t)kSlotsMaxChunks * kSlotsThreads);
  *chunk = (uint32_t)(std::max<int64_t>(c, 1) * kSlotsThreads);
  *chunks = (int)((pairs + *chunk - 1) / *chunk);
}

int launch_moe_slots(const SlotsArgs& a, hipStream_t s);
int launch_moe_combine(const CombineArgs& a, hipStream_t s);
int launch_moe_combine_bwd(const CombineArgs& a, hipStream_t s);
int launch_moe_route(const RouteArgs& a, hipStream_t s);
int launch_moe_route_bwd(const RouteBwdArgs& a, hipStream_t s);

}  // namespace hocf
