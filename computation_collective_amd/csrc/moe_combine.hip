// The weighted sum of the experts' rows and its gradients: nothing but
// memory traffic (a few flops for every 16 bytes), so every element is read
// and written once, in 16-byte pieces, with a token's rows all in flight
// together: 4096 tokens x 2 rows of 4096 bf16 from windows, with a residual,
// 25.4 us (5.3 TB/s), backward of 8191 x 8 x 2056 126 us (5.1 TB/s; a large copy
// reaches 5.0).
//
// Loads are unconditional (a pair without a row re-reads row 0, and the
// value is dropped, not multiplied by zero): a load under a condition becomes
// a branch and a full wait.
#include <algorithm>

#include "moe.hpp"
#include "sync.hpp"

namespace hocf {

constexpr int kCombineThreads = 256;
constexpr int64_t kMaxGrid = 1 << 23;  // workgroups of one launch (2^32 threads are too many)

// 16-byte accesses of what is read or written once and not used again soon.
typedef uint32_t uint32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint32x4 ld_once(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const uint32x4*>(p));
}
__device__ __forceinline__ void st_once(void* p, uint32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<uint32x4*>(p));
}

// Eight consecutive elements: as loaded, and as fp32.
template <int DT>
struct Raw8 {
  static constexpr int kPieces = DT == kBF16 ? 1 : 2;
  uint32x4 u[kPieces];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const char* q = reinterpret_cast<const char*>(p) + i * (DT == kBF16 ? 2 : 4);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) u[k] = ld_once(q + 16 * k);
  }
  __device__ __forceinline__ void load_again(const void* p, int64_t i) {  // (stays in the caches)
    const char* q = reinterpret_cast<const char*>(p) + i * (DT == kBF16 ? 2 : 4);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) u[k] = *reinterpret_cast<const uint32x4*>(q + 16 * k);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (DT == kBF16) f[k] = __uint_as_float(k & 1 ? u[0][k / 2] & 0xffff0000u : u[0][k / 2] << 16);
      else f[k] = __uint_as_float(u[k / 4 % kPieces][k % 4]);
    }
  }
};
template <int DT>
__device__ __forceinline__ void st8(void* p, int64_t i, const float (&f)[8]) {
  char* q = reinterpret_cast<char*>(p) + i * (DT == kBF16 ? 2 : 4);
  if constexpr (DT == kBF16) {
    st_once(q, uint32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])});
  } else {
#pragma unroll
    for (int k = 0; k < 8; k += 4)
      st_once(q + 4 * k, uint32x4{__float_as_uint(f[k]), __float_as_uint(f[k + 1]), __float_as_uint(f[k + 2]), __float_as_uint(f[k + 3])});
  }
}

// Row of place j of token t, or -1.
__device__ __forceinline__ int64_t row_of(const CombineArgs& a, int64_t t, int j) {
  if (!a.index) return t * a.topk + j;
  const int64_t r = a.index[t * a.topk + j];
  if (r >= -1 && r < a.R) return r;
  report_status(a.sync, kErrBadIndex);
  return -1;
}

// Forward: 1 << tx threads side by side on a token's pieces (the workgroup
// takes 256 >> tx tokens); blockIdx.y splits long rows.  K: the places held
// at once, 0 when there is no row at all (R == 0).
template <int DT, int ODT, int K>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(CombineArgs a, int tx) {
  const int N = a.N;
  for (int64_t t = ((int64_t)blockIdx.x << (8 - tx)) + (threadIdx.x >> tx); t < a.T; t += (int64_t)gridDim.x << (8 - tx)) {
    int64_t off[K > 0 ? K : 1];
    float w[K > 0 ? K : 1];
    bool live[K > 0 ? K : 1];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int jj = min(j, a.topk - 1);
      const int64_t r = row_of(a, t, jj);
      live[j] = j < a.topk && r >= 0;
      off[j] = max(r, (int64_t)0) * N;
      w[j] = a.weights[t * a.topk + jj];
    }
    if constexpr (K == 0)
      for (int j = 0; j < a.topk; ++j) (void)row_of(a, t, j);  // (reports an index that names a row)
    const int step = (int)(gridDim.y << tx) * 8;
    for (int n = (int)((blockIdx.y << tx) + (threadIdx.x & ((1u << tx) - 1))) * 8; n < N; n += step) {
      Raw8<DT> v[K > 0 ? K : 1];
      Raw8<ODT> r;
#pragma unroll
      for (int j = 0; j < K; ++j) v[j].load(a.rows, off[j] + n);
      if (a.add) r.load(a.add, t * N + n);
      float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < K; ++j) {
        float f[8];
        v[j].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = live[j] ? fmaf(w[j], f[i], s[i]) : s[i];
      }
      if (a.add) {
        float f[8];
        r.get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += f[i];
      }
      st8<ODT>(a.out, t * N + n, s);
    }
  }
}

// log2 of the threads that a row of `pieces` is given: the next power of two
// up to 256, at least 8.
static int row_threads(int64_t pieces, int most) {
  int tx = 3;
  while (tx < most && (int64_t(1) << tx) < pieces) ++tx;
  return tx;
}

template <int DT, int ODT, int K>
static int launch_fwd(const CombineArgs& a, hipStream_t s) {
  const int64_t pieces = a.N / 8;
  const int tx = row_threads(pieces, 8);
  const int64_t gx = (a.T + (kCombineThreads >> tx) - 1) / (kCombineThreads >> tx);
  const int gy = (int)std::max<int64_t>(1, std::min<int64_t>(pieces >> tx, 65535));
  hipLaunchKernelGGL((combine_kernel<DT, ODT, K>), dim3((uint32_t)std::min(gx, kMaxGrid), gy), dim3(kCombineThreads), 0, s, a, tx);
  return hipGetLastError();
}

template <int DT, int ODT>
static int launch_fwd_k(const CombineArgs& a, hipStream_t s) {
  if (a.R == 0) return launch_fwd<DT, ODT, 0>(a, s);
  switch (a.topk) {
    case 1: return launch_fwd<DT, ODT, 1>(a, s);
    case 2: return launch_fwd<DT, ODT, 2>(a, s);
    case 3: return launch_fwd<DT, ODT, 3>(a, s);
    case 4: return launch_fwd<DT, ODT, 4>(a, s);
    case 5: return launch_fwd<DT, ODT, 5>(a, s);
    case 6: return launch_fwd<DT, ODT, 6>(a, s);
    case 7: return launch_fwd<DT, ODT, 7>(a, s);
    case 8: return launch_fwd<DT, ODT, 8>(a, s);
  }
  return launch_fwd<DT, ODT, kRouteMaxTopk>(a, s);
}

int launch_moe_combine(const CombineArgs& a, hipStream_t s) {
  if (a.dt == kBF16) return a.out_dt == kBF16 ? launch_fwd_k<kBF16, kBF16>(a, s) : launch_fwd_k<kBF16, kF32>(a, s);
  return a.out_dt == kBF16 ? launch_fwd_k<kF32, kBF16>(a, s) : launch_fwd_k<kF32, kF32>(a, s);
}

// Backward.  The first workgroups zero the rows without a pair (kZeroRows
// rows each, from the inverse map); the others take a token each (4 waves on
// it) or a token per wave, read its dout and rows once, and write the rows'
// gradients and the dot products.
//
// Rows that are not whole cache lines (kShifted): a wave's pieces of each row
// start where the row's lines start, so that only a row's ends are written as
// parts of lines (8191 x 8 rows of 4112 bytes: 152 us unshifted, where rows of
// 4096 bytes take 134); dout is then read again at every row's pieces.  A dot product's partial sums fold in a
// fixed order (a lane's pieces, the lanes by halves, the waves in order).
constexpr int kZeroRows = 16;

template <int DT, int ODT, int K, BwdForm FORM>
__global__ __launch_bounds__(kCombineThreads) void combine_bwd_kernel(CombineArgs a, int64_t zero_blocks,
                                                                         int64_t blocks) {
  constexpr bool WIDE = FORM == kWide;
  constexpr int kPiece = 8 * (DT == kBF16 ? 2 : 4);  // bytes of a piece of a row
  __shared__ float s_dot[4][K];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int N = a.N;
  for (int64_t q = blockIdx.x; q < blocks; q += gridDim.x) {
    if (q < zero_blocks) {
      for (int i = wave; i < kZeroRows; i += 4) {
        const int64_t r = q * kZeroRows + i;
        if (r < a.R && a.pair[r] < 0) {
          const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int n = lane * 8; n < N; n += 512) st8<DT>(a.drows, r * N + n, z);
        }
      }
      continue;
    }
    const int64_t b = q - zero_blocks;
    const int64_t t = WIDE ? b : b * 4 + wave;
    if (t >= a.T) continue;  // (a whole wave, of a workgroup that meets at no barrier)
    int64_t off[K];
    float w[K], dot[K];
    bool live[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int jj = min(j, a.topk - 1);
      const int64_t r = row_of(a, t, jj);
      live[j] = j < a.topk && r >= 0;
      off[j] = max(r, (int64_t)0) * N;
      w[j] = a.weights[t * a.topk + jj];
      dot[j] = 0.0f;
    }
    if constexpr (FORM == kShifted) {
      int lead[K];  // elements from the line's start to the row's
#pragma unroll
      for (int j = 0; j < K; ++j)
        lead[j] = (int)((reinterpret_cast<uintptr_t>(a.drows) + off[j] * (kPiece / 8)) % kLine / kPiece) * 8;
      for (int n0 = lane * 8; n0 - lane * 8 < N + kLine / kPiece * 8 - 8; n0 += 64 * 8) {
        Raw8<DT> v[K];
        Raw8<ODT> d[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const int n = min(max(n0 - lead[j], 0), N - 8);
          d[j].load_again(a.dout, t * N + n);
          v[j].load(a.rows, off[j] + n);
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const int n = n0 - lead[j];
          if (!live[j] || n < 0 || n >= N) continue;
          float f[8], g[8], o[8];
          v[j].get(f);
          d[j].get(g);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(f[i], g[i], dot[j]);
            o[i] = w[j] * g[i];
          }
          st8<DT>(a.drows, off[j] + n, o);
        }
      }
    } else {
      for (int n = (WIDE ? (int)threadIdx.x : lane) * 8; n < N; n += (WIDE ? kCombineThreads : 64) * 8) {
        Raw8<DT> v[K];
        Raw8<ODT> d;
        d.load(a.dout, t * N + n);
        if (a.R > 0) {
#pragma unroll
          for (int j = 0; j < K; ++j) v[j].load(a.rows, off[j] + n);
        }
        float g[8];
        d.get(g);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          if (!live[j]) continue;
          float f[8], o[8];
          v[j].get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(f[i], g[i], dot[j]);
            o[i] = w[j] * g[i];
          }
          st8<DT>(a.drows, off[j] + n, o);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int d = 32; d; d >>= 1) dot[j] += __shfl_xor(dot[j], d, 64);
    if constexpr (WIDE) {
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < K; ++j) s_dot[wave][j] = dot[j];
      __syncthreads();
      if ((int)threadIdx.x < a.topk)
        a.dweights[t * a.topk + threadIdx.x] =
            s_dot[0][threadIdx.x] + s_dot[1][threadIdx.x] + s_dot[2][threadIdx.x] + s_dot[3][threadIdx.x];
      __syncthreads();  // (before the next item's)
    } else {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (lane == j && j < a.topk) a.dweights[t * a.topk + j] = dot[j];
    }
  }
}

template <int DT, int ODT, int K, BwdForm FORM>
static int launch_form(const CombineArgs& a, hipStream_t s) {
  const int64_t zero = a.pair ? (a.R + kZeroRows - 1) / kZeroRows : 0;
  const int64_t blocks = zero + (FORM == kWide ? a.T : (a.T + 3) / 4);
  hipLaunchKernelGGL((combine_bwd_kernel<DT, ODT, K, FORM>), dim3((uint32_t)std::min(blocks, kMaxGrid)),
                     dim3(kCombineThreads), 0, s, a, zero, blocks);
  return hipGetLastError();
}

template <int DT, int ODT, int K>
static int launch_bwd(const CombineArgs& a, hipStream_t s) {
  switch (combine_bwd_form(a.T, a.R, a.N, DT, reinterpret_cast<uintptr_t>(a.drows))) {
    case kWide: return launch_form<DT, ODT, K, kWide>(a, s);
    case kRows: return launch_form<DT, ODT, K, kRows>(a, s);
    default: return launch_form<DT, ODT, K, kShifted>(a, s);
  }
}

template <int DT, int ODT>
static int launch_bwd_k(const CombineArgs& a, hipStream_t s) {
  switch (a.topk) {
    case 1: return launch_bwd<DT, ODT, 1>(a, s);
    case 2: return launch_bwd<DT, ODT, 2>(a, s);
    case 3: return launch_bwd<DT, ODT, 3>(a, s);
    case 4: return launch_bwd<DT, ODT, 4>(a, s);
    case 5: return launch_bwd<DT, ODT, 5>(a, s);
    case 6: return launch_bwd<DT, ODT, 6>(a, s);
    case 7: return launch_bwd<DT, ODT, 7>(a, s);
    case 8: return launch_bwd<DT, ODT, 8>(a, s);
  }
  return launch_bwd<DT, ODT, kRouteMaxTopk>(a, s);
}

int launch_moe_combine_bwd(const CombineArgs& a, hipStream_t s) {
  if (a.dt == kBF16) return a.out_dt == kBF16 ? launch_bwd_k<kBF16, kBF16>(a, s) : launch_bwd_k<kBF16, kF32>(a, s);
  return a.out_dt == kBF16 ? launch_bwd_k<kF32, kBF16>(a, s) : launch_bwd_k<kF32, kF32>(a, s);
}

}  // namespace hocf
