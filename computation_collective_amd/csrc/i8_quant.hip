// Rows and weights to 8-bit codes, and back.
//
//   s = max(largest |x| / 127 (rounded to fp32), 2^-126),  q = x / s to the
//   nearest whole number, halves to the even one
// of the real quotient: bf16 rows meet halves often (x = m / 254 of the largest
// number), and a product with 1 / s would take them either way.  The product
// gives a candidate t; x - t s is a whole number of half steps of s's last bit
// and at most a little over s / 2, so an fma has it without error, and its size
// against s / 2 tells whether t stands.  (s is never subnormal, for its
// reciprocal and so that |q| stays below 128.)  A row with an infinity or a NaN
// gets the scale NaN and codes 0: what is computed from it is NaN.
//
// A row stays in registers between its largest number and its codes: read once.
// Bound by memory (8192 x 4096 bf16 20 us, 5.0 TB/s; reading 32768 x 1792 back 27 us,
// 6.4 TB/s with codes from the Infinity Cache), but for SiLU with both sides kept, whose
// vector instructions take as long (32768 x 1792: 49-58 us where memory would take 49).
#include <algorithm>

#include "i8.hpp"
#include "lanes.hpp"
#include "sync.hpp"

namespace hocf {

constexpr int kQThreads = 256;

// Workgroups in two dimensions (one dimension holds fewer than 2^32 threads), and a
// workgroup's number among them; those past the last have nothing to do.
static dim3 flat_grid(int64_t n) {
  const int64_t x = std::min<int64_t>(n, 1 << 20);
  return dim3((uint32_t)x, (uint32_t)((n + x - 1) / x));
}
__device__ __forceinline__ int64_t flat_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Eight consecutive numbers of a row, as loaded.
template <int DT>
struct Eight;
template <>
struct Eight<kBF16> {
  uint4 u;
  __device__ __forceinline__ void load(const void* row, int k) {
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    u = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(row) + k)));
  }
  __device__ __forceinline__ void load_cached(const void* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Eight<kF32> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const void* row, int k) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(row) + k);
    lo = p[0];
    hi = p[1];
  }
  __device__ __forceinline__ void load_cached(const void* p) { load(p, 0); }
  __device__ __forceinline__ float operator[](int i) const {
    const float4& q = i < 4 ? lo : hi;
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    lo = make_float4(v[0], v[1], v[2], v[3]);
    hi = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// The larger of the running magnitude and eight more: bits, in whose order NaN > infinity >
// numbers.  bf16: of pairs, side by side.
__device__ __forceinline__ uint32_t largest(const Eight<kF32>& e, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(e[i]) & 0x7fffffffu);
  return m;
}
typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t largest(const Eight<kBF16>& e, uint32_t m) {
  ushort2_t v = __builtin_bit_cast(ushort2_t, m);
  v = __builtin_elementwise_max(v, __builtin_bit_cast(ushort2_t, e.u.x & 0x7fff7fffu));
  v = __builtin_elementwise_max(v, __builtin_bit_cast(ushort2_t, e.u.y & 0x7fff7fffu));
  v = __builtin_elementwise_max(v, __builtin_bit_cast(ushort2_t, e.u.z & 0x7fff7fffu));
  v = __builtin_elementwise_max(v, __builtin_bit_cast(ushort2_t, e.u.w & 0x7fff7fffu));
  return __builtin_bit_cast(uint32_t, v);
}
// The bits of the larger of the pair, as fp32's.
template <int DT>
__device__ __forceinline__ uint32_t of_pair(uint32_t m) {
  return DT == kBF16 ? max(m & 0xffff0000u, m << 16) : m;
}

struct Scale {
  float s, inv;
  bool bad;
};
__device__ __forceinline__ Scale scale_of(uint32_t m) {
  Scale r;
  r.bad = m >= 0x7f800000u;
  r.s = fmaxf(__fdiv_rn(__uint_as_float(m), 127.0f), kI8TinyScale);
  r.inv = __frcp_rn(r.s);
  if (r.bad) r.s = __builtin_nanf("");
  return r;
}

// Eight codes.  1.5 * 2^23 + t has the byte t at its low end.
template <int DT>
__device__ __forceinline__ uint2 codes_of(const Eight<DT>& e, const Scale& sc) {
  constexpr float kMagic = 12582912.0f;
  float y[8], worst = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = fmaf(e[i], sc.inv, kMagic);
    worst = fmaxf(worst, fabsf(fmaf(kMagic - y[i], sc.s, e[i])));
  }
  if (worst + worst >= sc.s) {  // (a half, or a candidate on the wrong side of one; half the row's largest is one)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = fmaf(kMagic - y[i], sc.s, e[i]), d2 = fabsf(d) + fabsf(d);
      const int move = (int)(d2 > sc.s) | ((int)(d2 == sc.s) & (int)(__float_as_uint(y[i]) & 1u));
      y[i] += copysignf((float)move, d);
    }
  }
  auto four = [&](int i) {
    const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(y[i + 1]), __float_as_uint(y[i]), 0x0c0c0400u);
    const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(y[i + 3]), __float_as_uint(y[i + 2]), 0x04000c0cu);
    return ab | cd;
  };
  return sc.bad ? make_uint2(0, 0) : make_uint2(four(0), four(4));
}

// x / (1 + exp(-x)) of a number below -69, by a scaled exponent: its exp(x) may leave fp32's
// normal range while the result does not.  (Minus infinity gives NaN, as the quotient does.)
__device__ __forceinline__ float silu_far(float x) {
  return x * __builtin_amdgcn_exp2f(fmaf(x, 1.44269504f, 64.0f)) * 0x1p-64f;
}

// x / (1 + exp(-x)) rounded to bf16, in fp32: right for every one of the 65536 bf16 numbers (a test tries them all).
// The quotient's reciprocal gets a step of Newton's method, without which 5.9375 goes to the wrong side: it
// is 1.2 last bits of fp32 from a border of bf16's rounding, -3.046875 3.4 and the others 7 and more, where
// the error is 6.3 at most for |x| < 8 and grows with |x| (55 at -64, where no border is near).  2^-7 and -2^-8, less
// than 0.2 from a border, become the border itself, whose even side is theirs.
__device__ __forceinline__ Eight<kBF16> silu8(const Eight<kBF16>& e) {
  float v[8], t[8], far = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = e[i] * -1.44269504f;
    far = fmaxf(far, t[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = 1.0f + __builtin_amdgcn_exp2f(t[i]), inv = __builtin_amdgcn_rcpf(d), q = e[i] * inv;
    v[i] = fmaf(fmaf(-q, d, e[i]), inv, q);
  }
  if (far > 100.0f)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = silu_far(e[i]);
      v[i] = t[i] > 100.0f ? f : v[i];
    }
  Eight<kBF16> r;
  r.set(v);
  return r;
}
// In 64 bits for an fp32 result, whose last bit decides codes.
__device__ __forceinline__ Eight<kF32> silu8(const Eight<kF32>& e) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)((double)e[i] / (1.0 + exp(-(double)e[i])));
  Eight<kF32> r;
  r.set(v);
  return r;
}

template <int W, bool HALF>
__device__ __forceinline__ uint32_t row_largest(uint32_t m, uint32_t* s_max, int wave) {
  if constexpr (HALF) {
    uint32_t a, b;
    across<16>((uint32_t)row_max<16>((int)m), a, b);
    return max(a, b);
  }
  m = (uint32_t)row_max<64>((int)m);  // (magnitudes: the sign bit is clear)
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) s_max[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, s_max[w]);
  }
  return m;
}

// W waves a row (1 or 4), or HALF of one, up to C pieces of eight numbers a lane; LOOP: rows
// of any length, read twice.
// KEEP only with an activation: the codes of x and of act(x).
template <int DT, int ACT, bool KEEP, int W, int C, bool LOOP, bool HALF>
__global__ __launch_bounds__(kQThreads) void quant_kernel(QuantI8Args a) {
  __shared__ uint32_t s_max[2][4];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t row = HALF     ? flat_block() * 8 + wave * 2 + (lane >> 5)
                      : W == 1 ? flat_block() * 4 + wave
                               : flat_block();
  if (row >= a.T) return;  // (W = 4: the workgroup's row)
  const char* x = reinterpret_cast<const char*>(a.x) + row * a.ld * (DT == kBF16 ? 2 : 4);
  const int k0 = (HALF ? lane & 31 : W == 1 ? lane : (int)threadIdx.x) * 8;
  constexpr int kStep = HALF ? 256 : W * 512;
  static_assert(ACT == kSilu || !KEEP, "one side only");
  static_assert(!HALF || (W == 1 && !LOOP), "half of one wave");
  Eight<DT> v[LOOP ? 1 : C], p[KEEP && !LOOP ? C : 1];
  uint32_t m = 0, mp = 0;
  if constexpr (LOOP) {
    for (int k = k0; k < a.K; k += kStep) {
      Eight<DT> e;
      e.load(x, k);
      if constexpr (KEEP) mp = largest(e, mp);
      if constexpr (ACT == kSilu) e = silu8(e);
      m = largest(e, m);
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (k0 + c * kStep < a.K) (KEEP ? p[KEEP ? c : 0] : v[c]).load(x, k0 + c * kStep);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (k0 + c * kStep < a.K) {
        if constexpr (KEEP) {
          mp = largest(p[c], mp);
          v[c] = silu8(p[c]);
        } else if constexpr (ACT == kSilu) {
          v[c] = silu8(v[c]);
        }
        m = largest(v[c], m);
      }
  }
  const Scale s = scale_of(row_largest<W, HALF>(of_pair<DT>(m), s_max[0], wave));
  Scale sp = s;
  if constexpr (KEEP) sp = scale_of(row_largest<W, HALF>(of_pair<DT>(mp), s_max[1], wave));
  int8_t* q = a.codes + row * a.K;
  int8_t* qp = KEEP ? a.pre_codes + row * a.K : nullptr;
  auto put = [&](int k, const Eight<DT>& pre, const Eight<DT>& act) {
    *reinterpret_cast<uint2*>(q + k) = codes_of(act, s);
    if constexpr (KEEP) *reinterpret_cast<uint2*>(qp + k) = codes_of(pre, sp);
  };
  if constexpr (LOOP) {
    for (int k = k0; k < a.K; k += kStep) {
      Eight<DT> e;
      e.load(x, k);
      put(k, e, ACT == kSilu ? silu8(e) : e);
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (k0 + c * kStep < a.K) put(k0 + c * kStep, p[KEEP ? c : 0], v[c]);
  }
  if ((HALF ? (lane & 31) == 0 : lane == 0) && (W == 1 || wave == 0)) {
    a.scales[row] = s.s;
    if constexpr (KEEP) a.pre_scales[row] = sp.s;
  }
}

template <int DT, int ACT, bool KEEP, int W, int C, bool LOOP, bool HALF = false>
static int launch_q(const QuantI8Args& a, hipStream_t s) {
  const int64_t grid = HALF ? (a.T + 7) / 8 : W == 1 ? (a.T + 3) / 4 : a.T;
  hipLaunchKernelGGL((quant_kernel<DT, ACT, KEEP, W, C, LOOP, HALF>), flat_grid(grid), dim3(kQThreads), 0, s, a);
  return hipGetLastError();
}

// A wave a row where rows alone fill the device and fit a wave's registers (no barrier, and
// the next row's loads are another wave's), four waves a row else: a few rows' time is that of one.
template <int DT, int ACT, bool KEEP>
static int launch_act(const QuantI8Args& a, hipStream_t s) {
  if (a.T >= 2048 && a.K <= 4096) {
    // Half a wave a row where a whole one's last pass would be half empty, and what bounds the kernel is
    // vector instructions (bf16, SiLU with both sides, whole -> half a wave: 65536 x 768 55 -> 44 us,
    // 32768 x 1792 53 -> 49; 65536 x 256 without SiLU 18 -> 12).  Longer rows without SiLU are bound by
    // memory (32768 x 1792 32 -> 34), and of few a lane's time counts (2048 x 1792 6.8 -> 7.7).
    const bool half = a.K % 512 && a.K % 512 <= 256;
    if (half && a.K <= 1024) return launch_q<DT, ACT, KEEP, 1, 4, false, true>(a, s);
    if constexpr (ACT == kSilu)
      if (half && a.K <= 2048 && a.T >= 16384) return launch_q<DT, ACT, KEEP, 1, 8, false, true>(a, s);
    if (a.K <= 1024) return launch_q<DT, ACT, KEEP, 1, 2, false>(a, s);
    if (a.K <= 2048) return launch_q<DT, ACT, KEEP, 1, 4, false>(a, s);
    return launch_q<DT, ACT, KEEP, 1, 8, false>(a, s);
  }
  if (a.K <= 2048) return launch_q<DT, ACT, KEEP, 4, 1, false>(a, s);
  if (a.K <= 4096) return launch_q<DT, ACT, KEEP, 4, 2, false>(a, s);
  if (a.K <= 8192) return launch_q<DT, ACT, KEEP, 4, 4, false>(a, s);
  return launch_q<DT, ACT, KEEP, 4, 1, true>(a, s);
}
template <int DT>
static int launch_qdt(const QuantI8Args& a, hipStream_t s) {
  if (a.act == kSilu) return a.pre_codes ? launch_act<DT, kSilu, true>(a, s) : launch_act<DT, kSilu, false>(a, s);
  return launch_act<DT, kNone, false>(a, s);
}

int launch_quant_i8(const QuantI8Args& a, hipStream_t s) {
  return a.dt == kBF16 ? launch_qdt<kBF16>(a, s) : launch_qdt<kF32>(a, s);
}

// Reading back: 2^lg lanes take the pieces of eight codes of a row in turn.
template <int DT>
__global__ __launch_bounds__(kQThreads) void dequant_kernel(DequantI8Args a, int lg) {  // 2^lg lanes a row
  const int64_t i = flat_block() * kQThreads + threadIdx.x, row = i >> lg;
  if (row >= a.T) return;
  const float s = a.scales[row];
  for (int k = ((int)i & ((1 << lg) - 1)) * 8; k < a.K; k += 8 << lg) {
    const uint2 w = *reinterpret_cast<const uint2*>(a.codes + row * a.K + k);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3))) * s;
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    Eight<DT> r;
    r.set(v);
    u32x4_t* p = reinterpret_cast<u32x4_t*>(reinterpret_cast<char*>(a.out) + (row * a.K + k) * (DT == kBF16 ? 2 : 4));
    if constexpr (DT == kBF16) {
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, r.u), p);
    } else {
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, r.lo), p);
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, r.hi), p + 1);
    }
  }
}

int launch_dequant_i8(const DequantI8Args& a, hipStream_t s) {
  // a lane for every piece where there are few, up to a wave a row else
  const int most = a.T * a.K < (1 << 20) ? 13 : 6;
  int lg = 3;
  while (lg < most && (8 << lg) < a.K) ++lg;
  const int64_t grid = ((a.T << lg) + kQThreads - 1) / kQThreads;
  if (a.dt == kBF16) hipLaunchKernelGGL(dequant_kernel<kBF16>, flat_grid(grid), dim3(kQThreads), 0, s, a, lg);
  else hipLaunchKernelGGL(dequant_kernel<kF32>, flat_grid(grid), dim3(kQThreads), 0, s, a, lg);
  return hipGetLastError();
}

// Weights in two kernels.  First step: the largest magnitude of every column of a slab of rows.
// 64 columns x 256 rows a workgroup, eight lanes a row.
template <int DT>
__global__ __launch_bounds__(256) void w8_largest_kernel(WeightsI8Args a) {
  __shared__ uint32_t s_max[32][65];
  const int c8 = (threadIdx.x & 7) * 8, r0 = threadIdx.x >> 3;
  const int n = blockIdx.x * 64 + c8, e = blockIdx.z;
  uint32_t m[8] = {};
  if (n < a.N) {
    const int end = min(a.K, (int)(blockIdx.y + 1) * kW8SlabRows);
    for (int k = blockIdx.y * kW8SlabRows + r0; k < end; k += 32) {
      Eight<DT> v;
      v.load(reinterpret_cast<const char*>(a.W) + (((int64_t)e * a.K + k) * a.N + n) * (DT == kBF16 ? 2 : 4), 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = max(m[i], __float_as_uint(v[i]) & 0x7fffffffu);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s_max[r0][c8 + i] = m[i];
  __syncthreads();
  if (threadIdx.x < 64 && (int)(blockIdx.x * 64 + threadIdx.x) < a.N) {
    uint32_t t = 0;
    for (int r = 0; r < 32; ++r) t = max(t, s_max[r][threadIdx.x]);
    a.part[((int64_t)e * a.slabs + blockIdx.y) * a.N + blockIdx.x * 64 + threadIdx.x] = t;
  }
}

// Second step: 128 rows x 64 columns to codes, turned through LDS into 64 runs of 128 bytes.
template <int DT>
__global__ __launch_bounds__(256) void w8_codes_kernel(WeightsI8Args a) {
  __shared__ Scale s_scale[64];
  __shared__ __attribute__((aligned(16))) uint32_t s_q[64][36];  // [column][row / 4]: 144-byte rows
  const int e = blockIdx.z, n0 = blockIdx.x * 64, kb = blockIdx.y * 128;
  if (threadIdx.x < 64) {
    const int n = min(n0 + (int)threadIdx.x, a.N - 1);
    uint32_t m = 0;
    for (int j = 0; j < a.slabs; ++j) m = max(m, a.part[((int64_t)e * a.slabs + j) * a.N + n]);
    s_scale[threadIdx.x] = scale_of(m);
    if (blockIdx.y == 0 && n0 + (int)threadIdx.x < a.N) a.scales[(int64_t)e * a.N + n] = s_scale[threadIdx.x].s;
  }
  // four rows x eight columns a thread
  const int c8 = (threadIdx.x & 7) * 8, r4 = threadIdx.x >> 3;
  const int n = n0 + c8, k = kb + r4 * 4;
  Eight<DT> v[4];
  const bool mine = n < a.N && k < a.K;
  if (mine)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      v[r].load(reinterpret_cast<const char*>(a.W) + (((int64_t)e * a.K + k + r) * a.N + n) * (DT == kBF16 ? 2 : 4), 0);
  __syncthreads();
  if (mine) {
    // codes_of takes eight numbers with one scale: two columns' four rows share none, so a column at a time
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Scale sc = s_scale[c8 + i];
      Eight<kF32> col;
      const float f[8] = {v[0][i], v[1][i], v[2][i], v[3][i], 0.f, 0.f, 0.f, 0.f};
      col.set(f);
      s_q[c8 + i][r4] = codes_of(col, sc).x;
    }
  }
  __syncthreads();
  // 16 bytes a thread and pass: eight threads a column's 128 rows
#pragma unroll
  for (int t = threadIdx.x; t < 64 * 8; t += 256) {
    const int c = t >> 3, k16 = kb + (t & 7) * 16;
    if (n0 + c < a.N && k16 < a.K)
      *reinterpret_cast<uint4*>(a.wq + ((int64_t)e * a.N + n0 + c) * a.K + k16) =
          *reinterpret_cast<const uint4*>(&s_q[c][(t & 7) * 4]);
  }
}

// Both steps at once, for matrices of up to 512 P rows: 32 columns a workgroup, whose numbers
// stay in registers -- four rows x eight columns a thread and pass of 512 rows -- until their
// scales are known, and whose codes are turned in LDS.
template <int DT, int P>
__global__ __launch_bounds__(512) void w8_once_kernel(WeightsI8Args a) {
  constexpr int kRow = 512 * P + 16;  // bytes of a column's codes: columns start on different banks
  __shared__ __attribute__((aligned(16))) char s_q[32 * kRow];
  __shared__ uint32_t s_max[8][32];
  __shared__ Scale s_scale[32];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  // (the columns of an expert that share cache lines go to one XCD)
  const uint32_t b = xcd_contiguous(blockIdx.x, gridDim.x), nb = (a.N + 31) / 32;
  const int e = b / nb, n0 = (b - e * nb) * 32, c8 = (lane & 3) * 8, n = n0 + c8;
  const int r4 = (wave * 16 + (lane >> 2)) * 4;
  const char* w = reinterpret_cast<const char*>(a.W) + ((int64_t)e * a.K * a.N + min(n, a.N - 8)) * (DT == kBF16 ? 2 : 4);
  Eight<DT> v[P][4];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // (K is a multiple of 16: four rows are all there or none; rows past the last repeat it)
      const int k = min(p * 512 + r4 + r, a.K - 1);
      v[p][r].load_cached(w + (int64_t)k * a.N * (DT == kBF16 ? 2 : 4));
    }
  uint32_t m[8] = {};
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = max(m[i], __float_as_uint(v[p][r][i]) & 0x7fffffffu);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int d = 4; d < 64; d <<= 1) m[i] = max(m[i], (uint32_t)__shfl_xor((int)m[i], d, 64));
    if (lane < 4) s_max[wave][c8 + i] = m[i];
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    uint32_t t = 0;
    for (int i = 0; i < 8; ++i) t = max(t, s_max[i][threadIdx.x]);
    s_scale[threadIdx.x] = scale_of(t);
    if (n0 + (int)threadIdx.x < a.N) a.scales[(int64_t)e * a.N + n0 + threadIdx.x] = s_scale[threadIdx.x].s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Scale sc = s_scale[c8 + i];
#pragma unroll
    for (int p = 0; p < P; p += 2) {  // (two passes' four rows: eight numbers of one scale)
      const int q = p + 1 < P ? p + 1 : p;
      const float f[8] = {v[p][0][i], v[p][1][i], v[p][2][i], v[p][3][i], v[q][0][i], v[q][1][i], v[q][2][i], v[q][3][i]};
      Eight<kF32> col;
      col.set(f);
      const uint2 u = codes_of(col, sc);
      *reinterpret_cast<uint32_t*>(s_q + (c8 + i) * kRow + p * 512 + r4) = u.x;
      if (p + 1 < P) *reinterpret_cast<uint32_t*>(s_q + (c8 + i) * kRow + q * 512 + r4) = u.y;
    }
  }
  __syncthreads();
  const int pieces = a.K / 16;
  for (int t = threadIdx.x; t < 32 * pieces; t += 512) {
    const int c = t / pieces, k = (t - c * pieces) * 16;
    if (n0 + c < a.N)
      *reinterpret_cast<uint4*>(a.wq + ((int64_t)e * a.N + n0 + c) * a.K + k) = *reinterpret_cast<const uint4*>(s_q + c * kRow + k);
  }
}

template <int DT, int P>
static int launch_w8_once(const WeightsI8Args& a, hipStream_t s) {
  hipLaunchKernelGGL((w8_once_kernel<DT, P>), dim3((a.N + 31) / 32 * a.E), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <int DT>
static int launch_w8(const WeightsI8Args& a, hipStream_t s) {
  // One kernel where its workgroups are enough for most CUs (4 x 4096 x 1792 bf16, 224 of them: 27 us
  // against 36; 3 x 1040 x 1000 fp32, 96: 12.3 against 10.6) and K fits: a thread's share of more rows does
  // not fit its registers, nor the codes of 32 columns LDS.
  if ((a.N + 31) / 32 * a.E >= 160) {
    if (a.K <= 1024) return launch_w8_once<DT, 2>(a, s);
    if (a.K <= 2048) return launch_w8_once<DT, 4>(a, s);
    if constexpr (DT == kBF16)
      if (a.K <= 4096) return launch_w8_once<DT, 8>(a, s);
  }
  const int nb = (a.N + 63) / 64;
  hipLaunchKernelGGL(w8_largest_kernel<DT>, dim3(nb, a.slabs, a.E), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(w8_codes_kernel<DT>, dim3(nb, (a.K + 127) / 128, a.E), dim3(256), 0, s, a);
  return hipGetLastError();
}

int launch_weights_i8(const WeightsI8Args& a, hipStream_t s) {
  return a.dt == kBF16 ? launch_w8<kBF16>(a, s) : launch_w8<kF32>(a, s);
}

}  // namespace hocf
