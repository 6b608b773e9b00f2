// The rows of the combine's receive windows: pair i with bin b (the rank of
// its expert) has row b * cap + (earlier pairs of bin b).
//
// A wave takes 64 pairs at a time.  The ballots of the bits of their bins
// give, in a handful of instructions, the pairs of every bin (lane b counts
// bin b, so up to 64 bins) and each pair's rank among its bin's pairs of the
// wave; running counts, the counts of the workgroup's earlier waves and of
// earlier workgroups make that the pair's place.  No atomics: the places
// depend on the pairs alone.
//
// Two forms.  For few pairs, one kernel: every workgroup counts all the pairs,
// those before and after its own too, from one load of each.  Beyond, a kernel
// counts every chunk, and a second one sums the chunks before and after its own
// and places its pairs.  Both are bound by launches and latency (8192 pairs of 8
// bins 5.3 us, 524288 pairs of 16 bins 8.2 us), so everything a wave reads is on
// its way at once.
#include "lanes.hpp"
#include "moe.hpp"
#include "publish.hpp"
#include "sync.hpp"

namespace hocf {

constexpr int kSlotsWaves = kSlotsThreads / 64;

// The ballots of 64 pairs' bins, of NB bits (2^NB bins).
template <int NB>
struct BinBallots {
  uint64_t valid, bit[NB];
  __device__ __forceinline__ explicit BinBallots(int bin) {
    valid = __ballot(bin >= 0);
#pragma unroll
    for (int k = 0; k < NB; ++k) bit[k] = __ballot(bin >> k & 1);
  }
  // the lanes whose bin is b
  __device__ __forceinline__ uint64_t of(int b) const {
    uint64_t m = valid;
#pragma unroll
    for (int k = 0; k < NB; ++k) m &= (b >> k & 1) ? bit[k] : ~bit[k];
    return m;
  }
};

// x / d for quotients below 64 (d up to 2^31): a quotient in fp32, (x + 1/2) /
// d where that is exact, else put right.
struct SmallQuotient {
  uint32_t d;
  float inv;
  __device__ __forceinline__ explicit SmallQuotient(uint32_t d) : d(d), inv(1.0f / (float)d) {}
  __device__ __forceinline__ int operator()(uint32_t x) const {
    if (d < 1u << 15) return (int)fmaf((float)x, inv, 0.5f * inv);  // off by under 64 * 2^-22, 1/2d from a whole number
    int q = (int)((float)x * inv);
    const int32_t r = (int32_t)(x - (uint32_t)q * d);
    q -= r < 0;
    q += r >= (int32_t)d;
    return q;
  }
};

// Counts of up to 8 bins that a lane gathers by itself, 8 bits each (of up to 255
// pairs),
// and the wave's sums of them: a shift and an add a pair instead of ballots.
struct PackedCounts {
  uint64_t n = 0;
  __device__ __forceinline__ void add(int bin, bool yes = true) { n += bin >= 0 && yes ? 1ull << (8 * bin) : 0; }
  // lane b: the wave's pairs of bin b
  __device__ __forceinline__ uint32_t sums() const {
    const int lane = threadIdx.x & 63;
    uint32_t r = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t v = (uint32_t)(n >> (32 * h));
      const uint32_t even = row_add<64>(v & 0x00ff00ffu), odd = row_add<64>(v >> 8 & 0x00ff00ffu);  // (16 bits each)
      if (lane >> 2 == h) r = ((lane & 1 ? odd : even) >> (8 * (lane & 2))) & 0xffffu;
    }
    return r;
  }
};

// The experts of S strips of 64 pairs, `step` pairs apart (past the end: -1).
template <int S>
__device__ __forceinline__ void load_strips(const SlotsArgs& a, uint32_t begin, uint32_t step, uint32_t end, uint32_t (&e)[S]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 0; s < S; ++s) e[s] = a.experts[min(begin + s * step + lane, a.pairs - 1)];
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (begin + s * step + lane >= end) e[s] = ~0u;
}

__device__ __forceinline__ int bin_of(const SlotsArgs& a, const SmallQuotient& per_bin, uint32_t e) {
  return e < a.experts_end ? per_bin(e) : -1;
}

// Places S strips of pairs from `i0` on, `step` apart; base: the pairs of bin
// `lane` before them.
template <int NB, int S>
__device__ __forceinline__ void place_strips(const SlotsArgs& a, const int (&bin)[S], uint32_t i0, uint32_t step,
                                             uint32_t end, uint32_t base) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const uint32_t i = i0 + s * step + lane;
    const BinBallots<NB> bb(bin[s]);
    const uint64_t same = bb.of(bin[s]);
    const uint32_t first = __shfl(base, bin[s] & 63, 64);
    const uint32_t at = first + __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    const bool has = bin[s] >= 0 && at < a.cap;
    const uint32_t row = (uint32_t)bin[s] * a.cap + at;
    if (i < end) a.index[i] = has ? (int32_t)row : -1;
    if (has) a.pair[row] = (int32_t)i;
    base += (uint32_t)__popcll(bb.of(lane));
  }
}

// Rows without a pair: every workgroup fills its share of the rows.
__device__ __forceinline__ void fill_rest(const SlotsArgs& a, const uint32_t* s_total) {
  const uint32_t rows = (uint32_t)a.bins * a.cap;
  if (rows == 0) return;
  const SmallQuotient cap(a.cap);
  for (uint64_t r = (uint64_t)blockIdx.x * kSlotsThreads + threadIdx.x; r < rows; r += (uint64_t)gridDim.x * kSlotsThreads) {
    const int b = cap((uint32_t)r);
    if ((uint32_t)r - b * a.cap >= s_total[b]) a.pair[r] = -1;
  }
}

// One kernel, S strips of kSlotsThreads pairs; workgroup c places strip c.
template <int NB, int S>
__global__ __launch_bounds__(kSlotsThreads) void slots_direct_kernel(SlotsArgs a) {
  __shared__ uint32_t s_before[kSlotsWaves][64], s_all[kSlotsWaves][64], s_own[kSlotsWaves][64];
  __shared__ uint32_t s_total[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const SmallQuotient per_bin(a.per_bin);
  int mine[1] = {-1};
  uint32_t before = 0, own = 0, all = 0;
  if (a.pairs) {
    uint32_t e[S];
    load_strips<S>(a, wave * 64, kSlotsThreads, a.pairs, e);
    if constexpr (NB <= 3 && S > 1) {
      PackedCounts nb, na;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int bin = bin_of(a, per_bin, e[s]);
        na.add(bin);
        nb.add(bin, s < (int)blockIdx.x);
        if (s == (int)blockIdx.x) mine[0] = bin;
      }
      before = nb.sums();
      all = na.sums();
      own = (uint32_t)__popcll(BinBallots<NB>(mine[0]).of(lane));
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int bin = bin_of(a, per_bin, e[s]);
        const uint32_t n = (uint32_t)__popcll(BinBallots<NB>(bin).of(lane));
        all += n;
        if (s < (int)blockIdx.x) before += n;
        if (s == (int)blockIdx.x) { own = n; mine[0] = bin; }
      }
    }
  }
  s_before[wave][lane] = before;
  s_all[wave][lane] = all;
  s_own[wave][lane] = own;
  lds_barrier();
  uint32_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kSlotsWaves; ++w) {
    base += s_before[w][lane] + (w < wave ? s_own[w][lane] : 0u);
    total += s_all[w][lane];
  }
  if (wave == 0) {
    s_total[lane] = total;
    if (blockIdx.x == 0 && lane < a.bins) a.counts[lane] = total;
  }
  const uint32_t i0 = (uint32_t)blockIdx.x * kSlotsThreads + wave * 64;
  if (i0 < a.pairs) place_strips<NB, 1>(a, mine, i0, 64, a.pairs, base);
  lds_barrier();
  fill_rest(a, s_total);
}

// Chunks of S strips a wave: wave w has the pairs [w * S * 64, (w + 1) * S *
// 64) of its chunk.  Workspace: [chunk][2^NB] pairs of each bin.
template <int NB, int S>
__global__ __launch_bounds__(kSlotsThreads) void slots_count_kernel(SlotsArgs a) {
  __shared__ uint32_t s_n[kSlotsWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const SmallQuotient per_bin(a.per_bin);
  uint32_t n = 0;
  const uint32_t end = min(a.pairs, ((uint32_t)blockIdx.x + 1) * a.chunk);
  for (uint32_t i = (uint32_t)blockIdx.x * a.chunk + wave * (S * 64); i < end; i += kSlotsThreads * S) {
    uint32_t e[S];
    load_strips<S>(a, i, 64, end, e);
#pragma unroll
    for (int s = 0; s < S; ++s) n += (uint32_t)__popcll(BinBallots<NB>(bin_of(a, per_bin, e[s])).of(lane));
  }
  s_n[wave][lane] = n;
  lds_barrier();
  if (threadIdx.x < 1u << NB) {
    n = 0;
#pragma unroll
    for (int w = 0; w < kSlotsWaves; ++w) n += s_n[w][lane];
    a.hist[((int64_t)blockIdx.x << NB) + lane] = n;
  }
}

template <int NB, int S>
__global__ __launch_bounds__(kSlotsThreads) void slots_place_kernel(SlotsArgs a) {
  __shared__ uint32_t s_before[kSlotsWaves][64], s_all[kSlotsWaves][64], s_own[kSlotsWaves][64];
  __shared__ uint32_t s_total[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const SmallQuotient per_bin(a.per_bin);
  const uint32_t end = min(a.pairs, ((uint32_t)blockIdx.x + 1) * a.chunk);
  uint32_t i0 = (uint32_t)blockIdx.x * a.chunk + wave * (S * 64);
  uint32_t e[S];
  load_strips<S>(a, i0, 64, end, e);
  // the chunks' counts, 64 >> NB chunks a load: lane l has bin l mod 2^NB
  uint32_t before = 0, all = 0;
  const int words = a.chunks << NB, mine = blockIdx.x << NB;
  for (int k0 = wave * 64; k0 < words; k0 += kSlotsThreads * 4) {
    uint32_t n[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) n[u] = a.hist[min(k0 + u * kSlotsThreads + lane, words - 1)];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * kSlotsThreads + lane;
      all += k < words ? n[u] : 0u;
      before += k < mine ? n[u] : 0u;
    }
  }
  for (int d = 1 << NB; d < 64; d *= 2) {
    all += __shfl_xor(all, d, 64);
    before += __shfl_xor(before, d, 64);
  }
  // rounds of S strips a wave (one, unless there are more than kSlotsMaxChunks chunks' worth of pairs)
  uint32_t first = 0;  // pairs of bin `lane` in this chunk's earlier rounds
  for (bool again = false;; again = true) {
    int bin[S];
    uint32_t own = 0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      bin[s] = bin_of(a, per_bin, e[s]);
      own += (uint32_t)__popcll(BinBallots<NB>(bin[s]).of(lane));
    }
    if (again) lds_barrier();
    s_own[wave][lane] = own;
    if (!again) {
      s_before[wave][lane] = before;
      s_all[wave][lane] = all;
    }
    lds_barrier();
    uint32_t base = first, round = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kSlotsWaves; ++w) {
      const uint32_t o = s_own[w][lane];
      base += s_before[w][lane] + (w < wave ? o : 0u);
      round += o;
      total += s_all[w][lane];
    }
    first += round;
    if (wave == 0 && !again) {
      s_total[lane] = total;
      if (blockIdx.x == 0 && lane < a.bins) a.counts[lane] = total;
    }
    if (i0 < end) place_strips<NB, S>(a, bin, i0, 64, end, base);
    i0 += kSlotsThreads * S;
    if (i0 - wave * (S * 64) >= end) break;  // (the same in every wave)
    load_strips<S>(a, i0, 64, end, e);
  }
  lds_barrier();
  fill_rest(a, s_total);
}

template <int NB, int S>
static int launch_chunks(const SlotsArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((slots_count_kernel<NB, S>), dim3(a.chunks), dim3(kSlotsThreads), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((slots_place_kernel<NB, S>), dim3(a.chunks), dim3(kSlotsThreads), 0, s, a);
  return hipGetLastError();
}

template <int NB, int S>
static int launch_direct(const SlotsArgs& a, hipStream_t s) {
  const int grid = a.pairs ? (int)((a.pairs + kSlotsThreads - 1) / kSlotsThreads) : 1;
  hipLaunchKernelGGL((slots_direct_kernel<NB, S>), dim3(grid), dim3(kSlotsThreads), 0, s, a);
  return hipGetLastError();
}

// One kernel up to a workgroup's pairs, and with up to 8 bins up to eight:
// replayed from a graph, 8192 pairs take 5.2 us and the two kernels 5.6, 16384
// pairs 6.5 and 5.7 (called one by one, two launches take 8-9.5 us whatever they
// do).  With 16 bins the counts by ballots cost it more: 5.5 and 5.8 at 8192 pairs.
template <int NB>
static int launch_bits(const SlotsArgs& a, hipStream_t s) {
  if (a.pairs <= kSlotsThreads) return launch_direct<NB, 1>(a, s);
  if constexpr (NB <= 3) {
    if (a.pairs <= 4 * kSlotsThreads) return launch_direct<NB, 4>(a, s);
    if (a.pairs <= 8 * kSlotsThreads) return launch_direct<NB, 8>(a, s);
  }
  if (a.chunk <= kSlotsThreads) return launch_chunks<NB, 1>(a, s);
  if (a.chunk <= 2 * kSlotsThreads) return launch_chunks<NB, 2>(a, s);
  return launch_chunks<NB, 4>(a, s);
}

int launch_moe_slots(const SlotsArgs& a, hipStream_t s) {
  return a.bins <= 8 ? launch_bits<3>(a, s) : a.bins <= 16 ? launch_bits<4>(a, s) : launch_bits<6>(a, s);
}

}  // namespace hocf
