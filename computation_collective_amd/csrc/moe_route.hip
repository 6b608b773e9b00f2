// Routing to experts: the choice of every token's experts and their weights,
// and the gradient of the logits.
//
// Forward.  s = softmax(x) or sigmoid(x); v = s + bias; the best groups by
// the sum of their one or two largest v; the topk largest v of what is left,
// ties to the lower index; w = scale * s of the chosen, over their sum with
// renorm.
//
// A token has LPT lanes (16, or 64 where a lane's share would be too long);
// a lane holds a run of adjacent experts of one group.  The choice has to be
// the one that 64-bit scores make, but 64-bit scores for every expert cost
// more than everything else here, so it is made on 32-bit integer keys and
// kept only where they decide it:
//
//   key = v in fixed point, its low bits (Q units) replaced by the lane and the
//         slot within the lane (lower index, larger key), so that a token's keys
//         differ and the largest names its expert.
//   Order = kByLogit: without a bias, v rises with x, and v = x * 2^26 + 8.
//         Different keys (low bits aside) mean the same order of the scores:
//         the 8 puts the keys' borders where logits are 2^-47 apart or more,
//         and a logit's distance to the row's largest, below 64, is held to
//         2^-47.  So only equal keys are in doubt; equal keys of bf16 logits
//         that are not tiny are equal logits.
//   Order = kByScore: v = (s + bias) * 2^29.  A sigmoid in 32 bits is off by at
//         most 3.1 * 2^-24 (exponent, sum and reciprocal), a sum below 4 by 2
//         more, the conversion by one unit; a softmax by 35 * 2^-24 of the row's
//         largest score (a sum of up to 512 terms).  Neighbours nearer than that
//         allows are in doubt.
//
// A lane sorts its keys once; a choice is then the largest of the lanes' first
// keys, and its lane moves on by one.  The chosen keys go into a shift register
// across the lanes of 16, newest in lane 0, where what is in doubt is seen for
// all places at once.
//
// Neighbours in doubt are put in order by their exact values: a few more places
// are chosen until the next one is clearly below, the lanes evaluate the
// candidates' scores in 64 bits (a softmax's up to its sum) and rank them, equal
// ones by the lower index.  What that cannot settle (a group's
// place in doubt, a key outside the fixed-point range, a sigmoid beyond 20
// where 64 bits begin to saturate, a softmax with a bias) is chosen again in
// 64 bits by the whole wave: about 1e-4 of the tokens with biased sigmoids in
// groups, and of unit-normal logits without a bias none.  Rows that all need it
// (a chosen sigmoid beyond 20, a softmax's logit of 32 or more or 31 below zero
// among the chosen, more than 16 equal fp32 logits at the border) take five to
// seven times as long: 32768 tokens, 8 of 256, 75-100 us instead of 13-14.
//
// Bound by vector instructions, about 650 for a wave's four tokens of 256
// experts: 32768 tokens, top-8 of 256 with bias, groups and counts, 20-22 us
// (35.7 MB, 7 us at a large copy's rate), of them 12 us choosing, 4 us until
// the last wave's 64-bit choices are done, 2 us for the counts; 131072 tokens
// 54 us.
#include <algorithm>
#include <climits>

#include "lanes.hpp"
#include "moe.hpp"
#include "publish.hpp"
#include "sync.hpp"

namespace hocf {

constexpr int kRouteThreads = 512;
constexpr int kRouteWaves = kRouteThreads / 64;

enum Order : int { kByLogit, kByScore };
constexpr float kLogitUnit = 0x1p26f, kLogitShift = 8.0f, kScoreUnit = 0x1p29f;
// Twice the error of a score, in units of 2^-29 (and of a group's half sum of
// two scores, in units of 2^-28); the keys' low bits come on top.
constexpr int kDoubtSigmoid = 2 * 7 << 5, kDoubtSum = 2 * 3 << 5;
constexpr float kDoubtSoftmax = 2 * 36 << 5;  // times the largest score, and kDoubtSum
constexpr int kSaturated = 20 << 26;     // sigmoid(20) is 2e-9 from 1
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kVanished = -709.78f;    // a sigmoid below is 0 in 64 bits too
constexpr float kMaxF = 3.402823466e38f;

// A lane's keys in falling order: an odd-even merge sort, 63 exchanges of two
// instructions for 16 keys.
template <int W>
__device__ __forceinline__ void sort_falling(int (&k)[W]) {
#pragma unroll
  for (int p = 1; p < W; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < W; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < W && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const int hi = max(k[i + j], k[i + j + q]);
            k[i + j + q] = min(k[i + j], k[i + j + q]);
            k[i + j] = hi;
          }
}

// How a token's experts lie on its lanes.
struct Spread {
  int lg;       // log2 of the lanes of one group
  int run;      // experts of one lane
  int size;     // experts of one group
};

// Toward zero, saturating (-inf gives INT_MIN).
__device__ __forceinline__ int to_fixed(float f) {
  int r;
  __asm__("v_cvt_i32_f32 %0, %1" : "=v"(r) : "v"(f));
  return r;
}

// A logit as the operators take it: NaN as -inf, +inf as the largest number.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), kMaxF); }

// A lane's experts: `cnt` from expert `at` on, held in the W slots from expert
// `from` on (where at + W would leave the row, the slots start earlier, so
// that one load of W logits stays inside it; slots outside [lo, lo + cnt) are
// other lanes').
struct Run {
  int from, lo, cnt;
  __device__ __forceinline__ bool has(int i) const { return (uint32_t)(i - lo) < (uint32_t)cnt; }
};
template <int W>
__device__ __forceinline__ Run run_at(int at, int cnt, int E) {
  const int from = max(0, min(at, E - W));
  return Run{from, at - from, cnt};
}

// W adjacent elements as fp32, at any alignment.
template <int DT, int W>
__device__ __forceinline__ void load_row(const void* p, float (&x)[W]) {
  if constexpr (DT == kBF16) {
    if constexpr (W == 1) {
      x[0] = bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
    } else {
      uint32_t u[W / 2];
      __builtin_memcpy(u, p, sizeof u);
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    }
  } else {
    __builtin_memcpy(x, p, sizeof x);
  }
}

// A lane's logits, -inf in the slots that are not its own.
template <int DT, int W>
__device__ __forceinline__ void load_logits(const char* row, const Run& r, float (&x)[W]) {
  load_row<DT, W>(row + r.from * (DT == kBF16 ? 2 : 4), x);
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = clean(x[i]);
  if (!__all(r.cnt == W)) {
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = r.has(i) ? x[i] : -INFINITY;
  }
}

template <int CTRL>
__device__ __forceinline__ double dppd(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)u), hi = (uint32_t)dpp<CTRL>((int)(uint32_t)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int SWAP>
__device__ __forceinline__ double swapd(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  uint32_t lo[2], hi[2];
  across<SWAP>((uint32_t)u, lo[0], lo[1]);
  across<SWAP>((uint32_t)(u >> 32), hi[0], hi[1]);
  return fmax(__builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]), __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]));
}
__device__ __forceinline__ double wave_maxd(double v) {
  v = fmax(v, dppd<0xB1>(v));
  v = fmax(v, dppd<0x4E>(v));
  v = fmax(v, dppd<0x141>(v));
  v = fmax(v, dppd<0x140>(v));
  v = swapd<16>(v);
  return swapd<32>(v);
}

__device__ __forceinline__ double read_lane(double v, int lane) {  // (the same lane for the whole wave)
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Whether p holds in any lane of a token (16 or all 64).
template <int LPT>
__device__ __forceinline__ bool token_any(bool p) {
  const uint64_t b = __ballot(p);
  if (b == 0) return false;  // (the same in every lane)
  return LPT == 64 || (b >> (threadIdx.x & 48) & 0xffffu) != 0;
}

// A wave's room for a choice in 64 bits.
template <int N>
struct Room64 {
  double v[N];
  float bias[N];
};

// The choice of one token in 64 bits, by a whole wave (lane l: experts l, l +
// 64, ...; V of them); picks to LDS, -1 where none is left, and a softmax's
// largest logit and one over its sum.  Few tokens come here, but a wave that
// has one is the last to finish: it is laid out for a short chain of dependent
// steps and for little code, most of whose lines are fetched for this one token.
template <int DT, int V>
__device__ __forceinline__ void choose64(const RouteArgs& a, const void* row, double* lds, float* lds_bias, int* picks,
                                         float* top_out, float* inv_out) {
  const int lane = threadIdx.x & 63, E = a.E;
  const double kOff = -INFINITY;
  const bool softmax = a.score == kSoftmax;
  double top = -(double)kMaxF, sum = 0.0;
  {
    float x[V], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = min(lane + 64 * i, E - 1);
      x[i] = ld1<DT>(row, e);
      bias[i] = a.bias ? a.bias[e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = lane + 64 * i < E ? clean(x[i]) : -INFINITY;
      top = fmax(top, (double)x[i]);
      lds[lane + 64 * i] = x[i];
      lds_bias[lane + 64 * i] = bias[i];
    }
  }
  if (softmax) {
    top = wave_maxd(top);
    *top_out = (float)top;
  }
  uint32_t on = 0;
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    const double x = lds[lane + 64 * i], p = exp(softmax ? x - top : -x);
    on |= (uint32_t)(x > kOff) << i;
    lds[lane + 64 * i] = softmax ? p : 1.0 + p;
    sum += p;
  }
  if (softmax) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, 64);
    *inv_out = sum > 0.0 ? (float)(1.0 / sum) : 0.0f;
  }
  double v[V];
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    const double p = lds[lane + 64 * i];
    const double w = (softmax ? p : 1.0) / (softmax ? sum : p) + (double)lds_bias[lane + 64 * i];  // (sum = 0: every logit is off)
    lds[lane + 64 * i] = (on >> i & 1) && w > kOff ? w : kOff;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = lds[lane + 64 * i];
  if (a.n_group > 1) {
    // 1 << lg lanes on each group, strided through it
    const int size = E / a.n_group;
    int lg = 6;
    while ((64 >> lg) < a.n_group) --lg;
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    const int g = lane >> lg, step = 1 << lg;
    double m1 = kOff, m2 = kOff;
    if (g < a.n_group)
#pragma unroll 4
      for (int i = lane & (step - 1); i < size; i += step) {
        const double w = lds[g * size + i];
        m2 = fmax(m2, fmin(m1, w));
        m1 = fmax(m1, w);
      }
    auto merge = [&](double o1, double o2) {
      m2 = fmax(fmin(m1, o1), fmax(m2, o2));
      m1 = fmax(m1, o1);
    };
    if (step > 1) merge(dppd<0xB1>(m1), dppd<0xB1>(m2));
    if (step > 2) merge(dppd<0x4E>(m1), dppd<0x4E>(m2));
    if (step > 4) merge(dppd<0x141>(m1), dppd<0x141>(m2));
    if (step > 8) merge(dppd<0x140>(m1), dppd<0x140>(m2));
    if (step > 16) merge(__shfl_xor(m1, 16, 64), __shfl_xor(m2, 16, 64));  // (two groups at least)
    const double of = a.group_top == 2 && m2 > kOff ? m1 + m2 : m1;
    int ahead = 0;
#pragma unroll 4
    for (int o = 0; o < a.n_group; ++o) {
      const double other = read_lane(of, o << lg);
      ahead += other > of || (other == of && o < g);
    }
    const uint64_t kept = __ballot(g < a.n_group && ahead < a.topk_group);
    const float per = 1.0f / (float)size;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int of_e = min((int)(((float)(lane + 64 * i) + 0.5f) * per), a.n_group - 1);  // (lane + 64 i) / size
      if (!(kept >> (of_e << lg) & 1)) v[i] = kOff;
    }
  }
  int mine = -1;
  for (int j = 0; j < a.topk; ++j) {
    double best = v[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (v[i] > best) { best = v[i]; at = lane + 64 * i; }
    const double m = wave_maxd(best);
    const uint64_t who = __ballot(best == m);
    int e = __builtin_amdgcn_readlane(at, __builtin_ctzll(who));
    if (who & (who - 1)) {  // several: the lowest index
      int low = best == m ? at : INT_MAX;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) low = min(low, __shfl_xor(low, d, 64));
      e = uniform(low);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 64 * i == e) v[i] = kOff;
    if (lane == j) mine = m > kOff ? e : -1;
  }
  if (lane < a.topk) picks[lane] = mine;
}

// Counts of chosen experts leave a workgroup's LDS histogram through 64-bit
// words of the workspace: the high half counts the workgroups that have added,
// so that the last one to add an expert's word has its total, and no one waits
// for an order of separate additions.  Additions to one cache line go one
// after another (some 40 ns each, measured), so workgroups add to
// kCountCopies tables, and each table's last ones to a table of sums.  Every
// word is left zeroed by the last to add.
__device__ __forceinline__ bool add_counts(uint64_t* at, uint32_t n, uint32_t of, uint32_t* total) {
  const uint64_t was = __hip_atomic_fetch_add(at, (1ull << 32) + n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  *total = (uint32_t)was + n;
  const bool last = (uint32_t)(was >> 32) == of - 1;
  if (last) __hip_atomic_store(at, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return last;
}
__device__ __forceinline__ void finish_counts(const RouteArgs& a, const uint32_t* s_hist) {
  const uint32_t stride = route_count_stride(a.E), table = blockIdx.x % kCountCopies;
  const uint32_t groups = gridDim.x, of = (groups - table + kCountCopies - 1) / kCountCopies;  // that add to this table
  lds_barrier();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    uint32_t n;
    if (add_counts(&a.ws[(table + 1) * stride + e], s_hist[e], of, &n) &&
        add_counts(&a.ws[e], n, min(groups, (uint32_t)kCountCopies), &n))
      a.counts[e] = (int32_t)n;
  }
}

// A lane of a token has expert e (-1: none) of place `place` (outside [0, topk):
// nothing): its weight, and both to the outputs.  sigmoid(x) e^-c = e^(min(x, 0) - c) / (1 + e^-|x|);
// with renorm, c is the largest exponent, so that the sum cannot vanish.
template <int DT, int LPT>
__device__ __forceinline__ void emit(const RouteArgs& a, int64_t t, bool own, int place, int e, float top, float inv,
                                     uint32_t* hist) {
  const char* row = reinterpret_cast<const char*>(a.logits) + t * a.ld * (DT == kBF16 ? 2 : 4);
  const bool softmax = a.score == kSoftmax, has = (uint32_t)place < (uint32_t)a.topk;
  if (!has) e = -1;
  const float x = e >= 0 ? clean(ld1<DT>(row, e)) : -INFINITY;
  const float up = softmax ? x : fminf(x, 0.0f);
  float c = softmax ? top : 0.0f;
  if (a.renorm) c = fmaxf(row_maxf<LPT>(up), -kMaxF);
  float w = e >= 0 && (softmax || x >= kVanished) ? expf(up - c) : 0.0f;
  if (!softmax) {
    w /= 1.0f + expf(-fabsf(x));
    inv = 1.0f;
  }
  if (a.renorm) {
    const float sum = row_sum<LPT>(w);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  }
  if (has && own) {
    a.experts[t * a.topk + place] = e;
    a.weights[t * a.topk + place] = e >= 0 ? w * inv * a.scale : 0.0f;
    if (a.counts && e >= 0) atomicAdd(&hist[e], 1u);
  }
}

// A token whose candidates a wave has found but not ranked yet (n = 0: it has
// to be chosen in 64 bits).
struct Candidates {
  int64_t t;
  int n;
  float top, inv;
  int16_t e[kRouteMaxTopk];
};
constexpr int kWaveList = 8;       // of them, a wave (any more are marked in the output, to be chosen in 64 bits)
constexpr int kLater = INT_MIN;    // stands in a token's first place until it is chosen in 64 bits

template <int DT, int LPT, int W, Order ORDER>
__global__ __launch_bounds__(kRouteThreads, LPT == 64 ? 3 : W > 4 ? 4 : 6) void route_kernel(RouteArgs a, Spread sp) {
  constexpr int es = DT == kBF16 ? 2 : 4;
  constexpr int TPW = 64 / LPT;           // tokens of one wave
  constexpr int Q = LPT * W;              // units of a key that hold the lane and the slot
  constexpr int kLow = INT_MIN + Q;       // below: switched off (or far down)
  constexpr int kTop = INT_MAX & -Q;      // from here on: beyond the fixed-point range
  constexpr int kTiny = 512 * Q;          // below: bf16 neighbours can share a key
  constexpr bool kListed = W > 4;         // the lanes' sorted keys are in LDS, but for the first two
  // (one after the other: the keys, and the 64-bit values at the end)
  __shared__ union {
    Room64<LPT == 16 ? 256 : kRouteMaxE> exact;
    int keys[kListed ? W + 1 : 1][64];
  } s_wave[kRouteWaves];
  __shared__ int s_pick[kRouteWaves][kRouteMaxTopk];
  __shared__ Candidates s_list[kRouteWaves][kWaveList];
  __shared__ uint32_t s_hist[kRouteMaxE];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int l = lane & (LPT - 1), row_lane = lane & 15;
  // this lane's run of experts
  const int g = l >> sp.lg, in_group = (l & ((1 << sp.lg) - 1)) * sp.run;
  const int cnt = g < a.n_group ? min(max(sp.size - in_group, 0), sp.run) : 0;
  const Run mine = run_at<W>(cnt > 0 ? g * sp.size + in_group : 0, cnt, a.E);
  const bool softmax = a.score == kSoftmax;
  const int low_bits = (LPT - 1 - l) * W;

  // The 64-bit work waits until the wave's other tokens are done: here, its
  // registers (the exponential's constants above all) would halve the waves.
  int listed = 0;
  bool left = false;
  const int64_t begin = ((int64_t)blockIdx.x * kRouteWaves + wave) * TPW, step = (int64_t)gridDim.x * kRouteWaves * TPW;
  auto row_at = [&](int64_t t0) {  // (the wave's first row, and the lane's offset from it: up to 3 * 2^24 logits)
    const uint32_t off = (uint32_t)(min(t0 + lane / LPT, a.T - 1) - t0) * (uint32_t)a.ld;
    return reinterpret_cast<const char*>(a.logits) + t0 * a.ld * es + off * (uint32_t)es;
  };
  float x[W], bias[W];
  if (begin < a.T) load_row<DT, W>(row_at(begin) + mine.from * es, x);
  if constexpr (ORDER == kByScore) {
#pragma unroll
    for (int i = 0; i < W; ++i) bias[i] = 0.0f;
    if (a.bias) load_row<kF32, W>(a.bias + mine.from, bias);
  }
  if (a.counts) {
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) s_hist[e] = 0;
    lds_barrier();
  }
  if constexpr (ORDER == kByScore) {
#pragma unroll
    for (int i = 0; i < W; ++i) bias[i] = fmaxf(bias[i], -INFINITY) * kScoreUnit;  // (a NaN is as good as no expert)
  }
  for (int64_t t0 = begin; t0 < a.T; t0 += step) {
    // switched-off logits, and other lanes' slots
    bool live = mine.cnt == W;
#pragma unroll
    for (int i = 0; i < W; ++i) live &= x[i] > -INFINITY;
    const bool gaps = !__all(live);
    if (gaps) {
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = mine.has(i) && x[i] > -INFINITY ? x[i] : -INFINITY;
    }
    // softmax: the row's largest logit and sum
    float top = 0.0f, inv = 1.0f;
    if (softmax && (ORDER == kByScore || !a.renorm)) {
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = fminf(x[i], kMaxF);
      top = x[0];
#pragma unroll
      for (int i = 1; i < W; ++i) top = fmaxf(top, x[i]);
      top = fmaxf(row_maxf<LPT>(top), -kMaxF);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) sum += __builtin_amdgcn_exp2f((x[i] - top) * kLog2e);
      sum = row_sum<LPT>(sum);
      inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    const uint32_t unsure = softmax ? (uint32_t)(inv * kDoubtSoftmax) + kDoubtSum : kDoubtSigmoid;
    float v[W];
    if constexpr (ORDER == kByScore) {
      if (softmax) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = __builtin_amdgcn_exp2f((x[i] - top) * kLog2e) * inv;
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x[i] * kLog2e));
      }
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = fmaf(v[i], kScoreUnit, bias[i]);
      if (gaps) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = x[i] > -INFINITY ? v[i] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = fmaf(x[i], kLogitUnit, kLogitShift);
    }
    // the next tokens' logits are on their way during the choice
    if (t0 + step < a.T) load_row<DT, W>(row_at(t0 + step) + mine.from * es, x);
    int k[W];
#pragma unroll
    for (int i = 0; i < W; ++i) k[i] = (to_fixed(v[i]) & -Q) | (low_bits + W - 1 - i);
    sort_falling<W>(k);
    // to be chosen in 64 bits (the same in every lane of the token)
    bool hard = false;
    if (a.n_group > 1) {
      int m1 = k[0], m2 = W > 1 ? k[W > 1] : INT_MIN;
      auto merge = [&](int o1, int o2) {
        m2 = max(min(m1, o1), max(m2, o2));
        m1 = max(m1, o1);
      };
      if (sp.lg > 0) merge(dpp<0xB1>(m1), dpp<0xB1>(m2));
      if (sp.lg > 1) merge(dpp<0x4E>(m1), dpp<0x4E>(m2));
      if (sp.lg > 2) merge(dpp<0x141>(m1), dpp<0x141>(m2));
      if constexpr (LPT == 64) {
        if (sp.lg > 3) merge(dpp<0x140>(m1), dpp<0x140>(m2));
        if (sp.lg > 4) merge(__shfl_xor(m1, 16, 64), __shfl_xor(m2, 16, 64));
      }
      const bool group = g < a.n_group;
      int of = m1 & -Q, low_of = kLow;
      bool unclear = m1 >= kTop;
      if constexpr (ORDER == kByScore) {
        const bool two = a.group_top == 2 && sp.size > 1;
        of = (of >> 1) + (two && m2 >= kLow ? (m2 & -Q) >> 1 : 0);
        low_of = (kLow >> 1) + Q;
        unclear |= a.bias && (m1 < kLow || (two && m2 < kLow));
      }
      // one by one, the lower of equals first; the last that stays, and the first that does not
      of = group ? (of & -LPT) | (LPT - 1 - (l >> sp.lg << sp.lg)) : INT_MIN;
      bool kept = false;
      int in = 0;
      for (int j = 0; j < a.topk_group; ++j) {
        in = row_max<LPT>(of);
        const bool best = of == in;
        kept |= best;
        of = best ? INT_MIN : of;
      }
      const int out = row_max<LPT>(of);
      if (out > low_of) {
        if constexpr (ORDER == kByScore)
          hard = (uint32_t)in - (uint32_t)out < unsure + Q + 2 * LPT;
        else hard = ((in ^ out) & -LPT) == 0 && (DT != kBF16 || abs(in) < kTiny);
      }
      hard |= token_any<LPT>(group && unclear);
      if (!kept) {
#pragma unroll
        for (int i = 0; i < W; ++i) k[i] = INT_MIN;
      }
    }
    // The lanes' lists: the first key and the second, and where the third is.
    int* const last = &s_wave[wave].keys[kListed ? W : 0][lane];  // (always INT_MIN)
    const int* third = last;
    if constexpr (kListed) {
      __builtin_amdgcn_wave_barrier();  // (the wave is done with the last tokens' lists)
#pragma unroll
      for (int i = 2; i < W; ++i) s_wave[wave].keys[i][lane] = k[i];
      *last = INT_MIN;
      third = &s_wave[wave].keys[2][lane];
      __threadfence_block();
      __builtin_amdgcn_wave_barrier();
    }
    // The next choice: the largest of the first keys; its lane moves on.
    auto choose = [&] {
      if constexpr (kListed) {
        int after = *third;
        const int m = row_max<LPT>(k[0]);
        __asm__ volatile("" : "+v"(after));  // (read in time, not when it is needed)
        const bool winner = k[0] == m;
        k[0] = winner ? k[1] : k[0];
        k[1] = winner ? after : k[1];
        third += winner && third < last ? 64 : 0;
        return m;
      } else {
        const int m = row_max<LPT>(k[0]);
        const bool winner = k[0] == m;
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) k[i] = winner ? k[i + 1] : k[i];
        k[W - 1] = winner ? INT_MIN : k[W - 1];
        return m;
      }
    };
    auto shift_in = [&](int m, int q) { return __builtin_amdgcn_update_dpp(m, q, 0x111, 0xf, 0xf, false); };
    // Lane i of 16 has the choice of place n - 1 - i.
    int q = INT_MIN, n = 0;
    for (; n < a.topk; ++n) q = shift_in(choose(), q);
    int next = row_max<LPT>(k[0]);
    // whether two neighbours are in doubt (m the lower one)
    auto close = [&](int before, int m) {
      if (m < kLow) return false;
      if constexpr (ORDER == kByScore)
        return (uint32_t)(before & -Q) - (uint32_t)(m & -Q) < unsure + Q;
      else return ((before ^ m) & -Q) == 0 && (DT != kBF16 || abs(m) < kTiny);
    };
    bool doubt = row_lane < n && close(q, shift_in(next, q));
    const bool below = row_lane < n && q < kLow;  // the key of no live expert, or of one that is far down
    bool extreme = row_lane < n && (q >= kTop || (ORDER == kByLogit && !softmax && q > kSaturated));
    bool near = false;
    if (__any(doubt || below || extreme)) {
      if (ORDER == kByScore) extreme |= below && a.bias;
      else if (token_any<LPT>(below)) {
        float y[W];
        load_row<DT, W>(row_at(t0) + mine.from * es, y);
        bool down = false;
#pragma unroll
        for (int i = 0; i < W; ++i) down |= mine.has(i) && y[i] > -INFINITY && y[i] <= -31.0f;
        extreme |= token_any<LPT>(down);
      }
      hard |= token_any<LPT>(extreme);
      near = token_any<LPT>(doubt);
      // beyond the last place: as far as it is in doubt
      bool open = token_any<LPT>(doubt && row_lane == 0);
      while (__any(open)) {
        if (n == kRouteMaxTopk) {
          hard |= open;
          break;
        }
        const int m = choose();
        q = shift_in(m, q);
        ++n;
        next = row_max<LPT>(k[0]);
        open &= close(m, next);
      }
      if (ORDER == kByScore && softmax && a.bias) hard |= near;  // (exact values need the row's exact sum)
    }
    // the expert of a key: its lane and its slot
    const int of_lane = LPT - 1 - (int)((uint32_t)q / W & (LPT - 1));
    const int from = __shfl(mine.from, of_lane, LPT);
    const int place = row_lane < n && l < 16 ? n - 1 - row_lane : -1;
    const int e = place >= 0 && q >= kLow ? from + W - 1 - (q & (W - 1)) : -1;
    const int64_t t = min(t0 + lane / LPT, a.T - 1);
    const bool own = t0 + lane / LPT < a.T;
    if (__any(near || hard)) {
      // to the list, as far as there is room
      const uint64_t want = __ballot(l == 0 && own && (near || hard));
      const int at = listed + __builtin_popcountll(want & ((1ull << (lane & -LPT)) - 1));
      const bool listing = own && (near || hard) && at < kWaveList;
      if (listing) {
        Candidates& c = s_list[wave][at];
        if (l < kRouteMaxTopk) c.e[l] = (int16_t)e;
        if (l == 0) {
          c.t = t;
          c.n = hard ? 0 : n;
          c.top = top;
          c.inv = inv;
        }
      }
      const bool later = own && (near || hard) && !listing;
      if (later && l == 0) a.experts[t * a.topk] = kLater;
      listed = min(listed + (int)__builtin_popcountll(want), kWaveList);
      left |= __any(later);
    }
    emit<DT, LPT>(a, t, own && !near && !hard, place, e, top, inv, s_hist);
  }
  __threadfence_block();
  __builtin_amdgcn_wave_barrier();

  // Candidates: a lane each, ranked by their exact values, ties to the lower index.
  uint32_t whole = 0;
  for (int i0 = 0; i0 < listed; i0 += TPW) {
    const int at = i0 + lane / LPT;
    const Candidates& c = s_list[wave][min(at, listed - 1)];
    const int n = c.n, e = l < n ? c.e[min(l, kRouteMaxTopk - 1)] : -1;
    const bool own = at < listed && n > 0;
    const uint64_t none = __ballot(l == 0 && at < listed && n == 0);
    for (uint64_t u = none; u; u &= u - 1) whole |= 1u << (i0 + __builtin_ctzll(u) / LPT);
    if (!__any(own)) continue;
    const char* row = reinterpret_cast<const char*>(a.logits) + c.t * a.ld * es;
    const float x = e >= 0 ? clean(ld1<DT>(row, e)) : -INFINITY;
    // (the largest logit of a row is among the candidates where they are chosen by their logits)
    const float top = !softmax ? 0.0f : ORDER == kByLogit ? row_maxf<LPT>(x) : c.top;
    double v = exp(softmax ? (double)x - (double)top : -(double)x);
    if (!softmax) v = 1.0 / (1.0 + v);
    if (ORDER == kByScore && !softmax && a.bias && e >= 0) v += (double)a.bias[e];
    if (e < 0) v = -INFINITY;
    int rank = 0;
    for (int i = 0; i < kRouteMaxTopk; ++i) {
      const double o = __shfl(v, i, LPT);
      const int oe = __shfl(e, i, LPT);
      rank += i < n && (o > v || (o == v && (oe < e || (oe == e && i < l))));
    }
    emit<DT, LPT>(a, c.t, own, l < n ? rank : -1, e, c.top, c.inv, s_hist);
  }
  if (whole || left) {
    if (left) wait_memory();  // the marks are there
    int64_t t0 = begin;
    uint64_t todo = 0;  // marked tokens of the step before t0
    for (;;) {
      int64_t t;
      if (whole) {
        t = s_list[wave][__builtin_ctz(whole)].t;
        whole &= whole - 1;
      } else {
        for (; left && !todo && t0 < a.T; t0 += step) {
          const int mark = __hip_atomic_load(&a.experts[min(t0 + lane / LPT, a.T - 1) * a.topk], __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
          todo = __ballot(l == 0 && t0 + lane / LPT < a.T && mark == kLater);
        }
        if (!todo) break;
        t = t0 - step + __builtin_ctzll(todo) / LPT;
        todo &= todo - 1;
      }
      float top = 0.0f, inv = 1.0f;
      auto& room = s_wave[wave].exact;
      choose64<DT, LPT == 16 ? 4 : 8>(a, reinterpret_cast<const char*>(a.logits) + t * a.ld * es, room.v, room.bias,
                                      s_pick[wave], &top, &inv);
      __threadfence_block();
      __builtin_amdgcn_wave_barrier();
      emit<DT, LPT>(a, t, lane < LPT, l, s_pick[wave][min(l, kRouteMaxTopk - 1)], top, inv, s_hist);
      __builtin_amdgcn_wave_barrier();
    }
  }
  if (a.counts) finish_counts(a, s_hist);
}

template <int DT, int LPT, int W>
static int launch_route(const RouteArgs& a, const Spread& sp, hipStream_t s) {
  const bool by_score = a.bias || (a.n_group > 1 && a.group_top == 2);
  auto kern = by_score ? &route_kernel<DT, LPT, W, kByScore> : &route_kernel<DT, LPT, W, kByLogit>;
  int grid = 0;
  constexpr int64_t per = kRouteWaves * (64 / LPT);
  const hipError_t e = persistent_grid(reinterpret_cast<const void*>(kern), kRouteThreads, (a.T + per - 1) / per, &grid,
                                       a.counts ? 512 : 0);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kRouteThreads), 0, s, a, sp);
  return hipGetLastError();
}

static int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

template <int DT>
static int launch_route_dt(const RouteArgs& a, hipStream_t s) {
  Spread sp{};
  sp.size = a.E / a.n_group;
  const int groups = pow2_at_least(a.n_group);
  for (const int lpt : {16, 64}) {
    if (groups > lpt) continue;
    const int lanes = lpt / groups;
    sp.lg = __builtin_ctz(lanes);
    sp.run = (sp.size + lanes - 1) / lanes;
    if (lpt == 16) {
      if (sp.run <= 1) return launch_route<DT, 16, 1>(a, sp, s);
      if (sp.run <= 2) return launch_route<DT, 16, 2>(a, sp, s);
      if (sp.run <= 4) return launch_route<DT, 16, 4>(a, sp, s);
      if (sp.run <= 8) return launch_route<DT, 16, 8>(a, sp, s);
      if (sp.run <= 16) return launch_route<DT, 16, 16>(a, sp, s);
    } else {
      if (sp.run <= 8) return launch_route<DT, 64, 8>(a, sp, s);
      if (sp.run <= 16) return launch_route<DT, 64, 16>(a, sp, s);
    }
  }
  return kNoKernel;
}

int launch_moe_route(const RouteArgs& a, hipStream_t s) {
  return a.dt == kBF16 ? launch_route_dt<kBF16>(a, s) : launch_route_dt<kF32>(a, s);
}

// Backward.  With p the softmax of the row and g_j = scale * dw_j:
//   softmax:             dx_e = p_e (sum over j with e_j = e of g_j  -  sum_j p_{e_j} g_j)
//   sigmoid:             dx_{e_j} = g_j s (1 - s), zero elsewhere
//   either with renorm:  w = scale * r with r the softmax of the chosen
//                        log-scores l_j, so d/dl_j = r_j (g_j - sum_k r_k g_k);
//                        l = x up to a constant for a softmax, log s for a
//                        sigmoid (dl/dx = 1 - s); zero elsewhere
// The log-score form keeps renorm exact where every chosen s underflows.
// A token has 16 lanes; lane j holds place j, and its contribution reaches
// the lane that holds expert e_j through an LDS row of the token.
constexpr int kBwdThreads = 256;
constexpr int kBwdTokens = kBwdThreads / 16;

// A lane's own elements: W at once, at any alignment, where all are its own.
template <int DT, int W>
__device__ __forceinline__ void store_row(char* row, const Run& r, const float (&d)[W]) {
  constexpr int es = DT == kBF16 ? 2 : 4;
  if (r.cnt == W) {
    char* p = row + r.from * es;
    if constexpr (DT == kBF16 && W > 1) {
      uint32_t u[W / 2];
#pragma unroll
      for (int i = 0; i < W; i += 2) u[i / 2] = pack_bf16x2(d[i], d[i + 1]);
      __builtin_memcpy(p, u, sizeof u);
    } else if constexpr (DT == kBF16) {
      st1<DT>(p, 0, d[0]);
    } else {
      __builtin_memcpy(p, d, sizeof d);
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (r.has(i)) st1<DT>(row, r.from + i, d[i]);
  }
}

template <int DT, int W>
__global__ __launch_bounds__(kBwdThreads) void route_bwd_kernel(RouteBwdArgs a, int run) {
  __shared__ __attribute__((aligned(16))) float s_d[kBwdTokens][16 * W];
  constexpr int es = DT == kBF16 ? 2 : 4;
  const int l = threadIdx.x & 15;
  float* mine = s_d[threadIdx.x >> 4];
  const int cnt = min(max(a.E - l * run, 0), run);
  const Run held = run_at<W>(cnt > 0 ? l * run : 0, cnt, a.E);
  const int per_run = 65536 / run + 1;  // (exact for e < 512, run <= 32)
  const bool softmax = a.score == kSoftmax, dense = softmax && !a.renorm;
  const int64_t step = (int64_t)gridDim.x * kBwdTokens;
  for (int64_t t0 = (int64_t)blockIdx.x * kBwdTokens + (threadIdx.x >> 6) * 4; t0 < a.T; t0 += step) {
    const int64_t tt = t0 + (threadIdx.x >> 4 & 3), t = min(tt, a.T - 1);
    const char* row = reinterpret_cast<const char*>(a.logits) + t * a.ld * es;
    float p[W];
    if (dense) load_logits<DT, W>(row, held, p);
    // lane j: place j
    int e = -1;
    float x = -INFINITY, g = 0.0f;
    if (l < a.topk) {
      e = a.experts[t * a.topk + l];
      if (e < -1 || e >= a.E) { report_status(a.sync, kErrBadIndex); e = -1; }
      if (e >= 0) {
        x = clean(ld1<DT>(row, e));
        if (x > -INFINITY) g = a.dweights[t * a.topk + l] * a.scale;
        if (x == -INFINITY || (!softmax && x < kVanished)) e = -1;  // a switched-off logit has no gradient
      }
    }
    float top = 0.0f, inv = 0.0f, mean = 0.0f, d = 0.0f;
    if (dense) {
      top = p[0];
#pragma unroll
      for (int i = 1; i < W; ++i) top = fmaxf(top, p[i]);
      top = fmaxf(row_maxf<16>(top), -kMaxF);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        p[i] = __builtin_amdgcn_exp2f((p[i] - top) * kLog2e);
        sum += p[i];
      }
      sum = row_sum<16>(sum);
      inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      d = g;
      mean = row_sum<16>(e >= 0 ? __builtin_amdgcn_exp2f((x - top) * kLog2e) * inv * g : 0.0f);
    } else {
      const float far = expf(-fabsf(x)), s0 = 1.0f / (1.0f + far);  // sigmoid(|x|)
      const float s1 = far * s0;                                    // 1 - sigmoid(|x|)
      const float s = x >= 0.0f ? s0 : s1, c = x >= 0.0f ? s1 : s0; // sigmoid(x), 1 - sigmoid(x)
      if (a.renorm) {
        const float up = softmax ? x : fminf(x, 0.0f);
        const float most = fmaxf(row_maxf<16>(e >= 0 ? up : -INFINITY), -kMaxF);
        float r = e >= 0 ? expf(up - most) * (softmax ? 1.0f : s0) : 0.0f;
        const float sum = row_sum<16>(r);
        r = sum > 0.0f ? r / sum : 0.0f;
        d = r * (g - row_sum<16>(r * g)) * (softmax ? 1.0f : c);
      } else {
        d = g * s * c;
      }
    }
    // to the lanes that hold the experts (places that name one expert twice add up)
#pragma unroll
    for (int i = 0; i < W; ++i) mine[i * 16 + l] = 0.0f;
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    const int holder = e * per_run >> 16;  // e / run
    if (e >= 0) atomicAdd(&mine[(e - max(0, min(holder * run, a.E - W))) * 16 + holder], d);
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    float o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      o[i] = mine[i * 16 + l];
      if (dense) o[i] = p[i] > 0.0f ? p[i] * inv * (o[i] - mean) : 0.0f;
    }
    __builtin_amdgcn_wave_barrier();
    if (tt < a.T) store_row<DT, W>(reinterpret_cast<char*>(a.dlogits) + t * a.E * es, held, o);
  }
}

template <int DT, int W>
static int launch_bwd(const RouteBwdArgs& a, hipStream_t s) {
  const int run = (a.E + 15) / 16;
  auto kern = &route_bwd_kernel<DT, W>;
  int grid = 0;
  const hipError_t e = persistent_grid(reinterpret_cast<const void*>(kern), kBwdThreads,
                                       (a.T + kBwdTokens - 1) / kBwdTokens, &grid);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kBwdThreads), 0, s, a, run);
  return hipGetLastError();
}

template <int DT>
static int launch_bwd_dt(const RouteBwdArgs& a, hipStream_t s) {
  const int run = (a.E + 15) / 16;
  if (run <= 1) return launch_bwd<DT, 1>(a, s);
  if (run <= 2) return launch_bwd<DT, 2>(a, s);
  if (run <= 4) return launch_bwd<DT, 4>(a, s);
  if (run <= 8) return launch_bwd<DT, 8>(a, s);
  if (run <= 16) return launch_bwd<DT, 16>(a, s);
  return launch_bwd<DT, 32>(a, s);
}

int launch_moe_route_bwd(const RouteBwdArgs& a, hipStream_t s) {
  return a.dt == kBF16 ? launch_bwd_dt<kBF16>(a, s) : launch_bwd_dt<kF32>(a, s);
}

}  // namespace hocf
