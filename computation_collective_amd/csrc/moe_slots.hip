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
// Two forms.  Up to kSlotsDirectPairs pairs, one kernel: every workgroup
// counts all the pairs before and after its own itself.  Beyond, a kernel
// counts every chunk, and a second one sums the chunks before and after its
// own and places its pairs.
#include "moe.hpp"
#include "sync.hpp"

namespace hocf {

constexpr int kSlotsWaves = kSlotsThreads / 64;
constexpr uint32_t kSlotsDirectPairs = 16384;

// The ballots of 64 pairs' bins.
struct BinBallots {
  uint64_t valid, bit[6];
  __device__ __forceinline__ BinBallots(int bin, int nb) {
    valid = __ballot(bin >= 0);
#pragma unroll
    for (int k = 0; k < 6; ++k) bit[k] = k < nb ? __ballot(bin >> k & 1) : 0;
  }
  // the lanes whose bin is b (b < 2^nb)
  __device__ __forceinline__ uint64_t of(int b, int nb) const {
    uint64_t m = valid;
#pragma unroll
    for (int k = 0; k < 6; ++k)
      if (k < nb) m &= (b >> k & 1) ? bit[k] : ~bit[k];
    return m;
  }
};

__device__ __forceinline__ int load_bin(const SlotsArgs& a, uint32_t i, uint32_t end) {
  const uint32_t e = i < end ? (uint32_t)a.experts[i] : ~0u;
  return e < a.experts_end ? (int)(e / (uint32_t)a.per_bin) : -1;
}

__device__ __forceinline__ int bits_of(int bins) { return bins > 1 ? 32 - __builtin_clz(bins - 1) : 0; }

// Lane b: pairs of bin b among [begin, end), begin a multiple of 64.
__device__ __forceinline__ uint32_t count_run(const SlotsArgs& a, uint32_t begin, uint32_t end, uint32_t step, int nb) {
  const int lane = threadIdx.x & 63;
  uint32_t n = 0;
  for (uint32_t i = begin; i < end; i += step)
    n += (uint32_t)__popcll(BinBallots(load_bin(a, i + lane, end), nb).of(lane, nb));
  return n;
}

__global__ __launch_bounds__(kSlotsThreads) void slots_count_kernel(SlotsArgs a) {
  __shared__ uint32_t s_n[kSlotsWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t begin = (uint32_t)blockIdx.x * a.chunk, end = min(a.pairs, begin + a.chunk);
  s_n[wave][lane] = count_run(a, begin + wave * 64, end, kSlotsThreads, bits_of(a.bins));
  __syncthreads();
  if (threadIdx.x < 64) {
    uint32_t n = 0;
    for (int w = 0; w < kSlotsWaves; ++w) n += s_n[w][lane];
    a.hist[(int64_t)blockIdx.x * 64 + lane] = n;
  }
}

template <bool DIRECT>
__global__ __launch_bounds__(kSlotsThreads) void slots_place_kernel(SlotsArgs a) {
  __shared__ uint32_t s_before[kSlotsWaves][64], s_rest[kSlotsWaves][64], s_own[kSlotsWaves][64];
  __shared__ uint32_t s_total[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nb = bits_of(a.bins);
  const uint32_t begin = min(a.pairs, (uint32_t)blockIdx.x * a.chunk), end = min(a.pairs, begin + a.chunk);
  // pairs of every bin before and after this chunk, a share per wave
  if constexpr (DIRECT) {
    s_before[wave][lane] = count_run(a, wave * 64, begin, kSlotsThreads, nb);
    s_rest[wave][lane] = count_run(a, end + wave * 64, a.pairs, kSlotsThreads, nb);
  } else {
    uint32_t before = 0, rest = 0;
    for (int c = wave; c < a.chunks; c += kSlotsWaves) {
      const uint32_t n = a.hist[(int64_t)c * 64 + lane];
      if (c < (int)blockIdx.x) before += n;
      else if (c > (int)blockIdx.x) rest += n;
    }
    s_before[wave][lane] = before;
    s_rest[wave][lane] = rest;
  }
  // this chunk: wave w has the pairs [begin + w * run, begin + (w + 1) * run)
  const uint32_t run = a.chunk / kSlotsWaves;
  const uint32_t mine = min(end, begin + wave * run), mine_end = min(end, mine + run);
  s_own[wave][lane] = count_run(a, mine, mine_end, 64, nb);
  __syncthreads();
  uint32_t base = 0, total = 0;
  for (int w = 0; w < kSlotsWaves; ++w) {
    base += s_before[w][lane] + (w < wave ? s_own[w][lane] : 0u);
    total += s_before[w][lane] + s_rest[w][lane] + s_own[w][lane];
  }
  if (wave == 0) {
    s_total[lane] = total;
    if (blockIdx.x == 0 && lane < a.bins) a.counts[lane] = total;
  }
  for (uint32_t i0 = mine; i0 < mine_end; i0 += 64) {
    const uint32_t i = i0 + lane;
    const int bin = load_bin(a, i, mine_end);
    const BinBallots bb(bin, nb);
    const uint64_t same = bb.of(bin, nb);
    const uint32_t first = __shfl(base, bin & 63, 64);
    const uint32_t at = first + __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    const bool has = bin >= 0 && at < a.cap;
    const uint32_t row = (uint32_t)bin * a.cap + at;
    if (i < mine_end) a.index[i] = has ? (int32_t)row : -1;
    if (has) a.pair[row] = (int32_t)i;
    base += (uint32_t)__popcll(bb.of(lane, nb));
  }
  __syncthreads();
  // rows without a pair: every workgroup fills its share of the rows
  const uint32_t rows = (uint32_t)a.bins * a.cap;
  for (uint64_t r = (uint64_t)blockIdx.x * kSlotsThreads + threadIdx.x; r < rows; r += (uint64_t)gridDim.x * kSlotsThreads) {
    const uint32_t b = (uint32_t)r / a.cap;
    if ((uint32_t)r - b * a.cap >= s_total[b]) a.pair[r] = -1;
  }
}

int launch_moe_slots(const SlotsArgs& args, hipStream_t s) {
  SlotsArgs a = args;
  if (a.pairs <= kSlotsDirectPairs) {
    a.chunk = kSlotsThreads;
    const int grid = a.pairs ? (int)((a.pairs + a.chunk - 1) / a.chunk) : 1;
    hipLaunchKernelGGL(slots_place_kernel<true>, dim3(grid), dim3(kSlotsThreads), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(slots_count_kernel, dim3(a.chunks), dim3(kSlotsThreads), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(slots_place_kernel<false>, dim3(a.chunks), dim3(kSlotsThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace hocf
