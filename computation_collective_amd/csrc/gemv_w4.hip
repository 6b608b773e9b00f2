// Products of a few token rows with their experts' 4-bit weights.
//
// The weights stream from HBM once; everything else (x, scales) is small.  A
// block of 128 rows x 16 columns is one 16-byte load per lane, laid out as
// the B operand of four 16x16x32 bf16 matrix products (lane q * 16 + n: column
// n, rows 32 t + 8 q + i of word t), with up to 16 token rows as the A
// operand.  A rotation and one mask turn eight codes into the bf16 numbers
// 16 + code; with sx = sum of x over a group (a product with ones),
//   sum x (code - zero) = sum x (16 + code)  -  (16 + zero) sx
// in fp32, then times the group's scale.
//
// A workgroup takes one block of 16 columns of one expert; its four waves
// take every fourth block of rows and fold through LDS in a fixed order.
#include <algorithm>

#include "moe.hpp"
#include "sync.hpp"

namespace hocf {

constexpr int kW4Threads = 256;
constexpr int kW4Waves = kW4Threads / 64;

// Eight codes of one packed word as 16 + code, in row order.
__device__ __forceinline__ bf16x8 codes_plus16(uint32_t w) {
  uint4 r;
  r.x = (w & 0x00780078u) | 0x41804180u;
  r.y = (__builtin_amdgcn_alignbit(w, w, 4) & 0x00780078u) | 0x41804180u;
  r.z = (__builtin_amdgcn_alignbit(w, w, 8) & 0x00780078u) | 0x41804180u;
  r.w = (__builtin_amdgcn_alignbit(w, w, 12) & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(bf16x8, r);
}

// Row r's expert among this rank's, or -1.
__device__ __forceinline__ int local_expert(const GemvW4Args& a, int r) {
  const uint32_t e = (uint32_t)a.experts[r] - (uint32_t)a.e0;
  return e < (uint32_t)a.E ? (int)e : -1;
}

template <int ODT, int GROUP, bool ZEROS>
__global__ __launch_bounds__(kW4Threads) void gemv_w4_kernel(GemvW4Args a, bool by_row) {
  __shared__ uint16_t s_rows[kW4MaxRows];
  __shared__ int s_n;
  __shared__ float s_part[kW4Waves][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cb = blockIdx.x, y = blockIdx.y;
  // this workgroup's expert: the y-th local one, or row y's (and then only
  // for the first of the rows that chose it)
  const int want = !a.experts ? 0 : by_row ? local_expert(a, y) : y;
  if (wave == 0) {
    int n = 0;
    bool first = true;
    for (int r0 = 0; r0 < a.R; r0 += 64) {
      const int r = r0 + lane;
      const int e = r >= a.R ? -1 : a.experts ? local_expert(a, r) : 0;
      const bool mine = r < a.R && e >= 0 && e == want;
      const uint64_t m = __ballot(mine);
      if (by_row && m && n == 0 && r0 + __builtin_ctzll(m) < y) first = false;
      if (mine) s_rows[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0))] = (uint16_t)r;
      n += __popcll(m);
      // rows of other ranks' experts: zeros, by the row's own workgroup or the first expert's
      if (a.experts && e < 0 && r < a.R && (by_row ? r == y : y == 0))
        for (int c = cb * 16; c < min(a.N, cb * 16 + 16); ++c) st1<ODT>(a.out, (int64_t)r * a.N + c, 0.0f);
    }
    if (lane == 0) s_n = first ? n : 0;
  }
  __syncthreads();
  const int n_rows = uniform(s_n);
  if (n_rows == 0) return;

  constexpr int WPG = GROUP / 32;  // words of one group
  const int q = lane >> 4, c = lane & 15;
  const uint4* w = reinterpret_cast<const uint4*>(a.wq) + ((int64_t)want * a.nb + cb) * a.kb * 64 + lane;
  const uint16_t* sc = a.scales + ((int64_t)want * a.nb + cb) * a.groups * 16 + c;
  const uint16_t* zp = ZEROS ? a.zeros + ((int64_t)want * a.nb + cb) * a.groups * 16 + c : nullptr;
  bf16x8 ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;

  for (int r0 = 0; r0 < n_rows; r0 += 16) {
    // A operand: lane's token row c (rows past the last repeat it, unused) at k = 32 t + 8 q
    const int row = s_rows[min(r0 + c, n_rows - 1)];
    const uint16_t* x = a.x + (int64_t)(row / a.rows_per_x) * a.K;
    floatx4 total = {0.f, 0.f, 0.f, 0.f};
    for (int kb = wave; kb < a.kb; kb += kW4Waves) {
      const uint4 wv = w[(int64_t)kb * 64];
      const uint32_t word[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int g = 0; g < 4 / WPG; ++g) {
        const int gi = min((kb * 128 + g * GROUP) / GROUP, a.groups - 1);
        const float s = bf16_to_f32(sc[gi * 16]);
        const float z = 16.0f + (ZEROS ? bf16_to_f32(zp[gi * 16]) : 8.0f);
        floatx4 acc = {0.f, 0.f, 0.f, 0.f}, sx = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = g * WPG; t < (g + 1) * WPG; ++t) {
          const int k = kb * 128 + t * 32 + q * 8;
          uint4 xv = *reinterpret_cast<const uint4*>(x + min(k, a.K - 8));
          if (k >= a.K) xv = make_uint4(0, 0, 0, 0);  // rows beyond K
          const bf16x8 av = __builtin_bit_cast(bf16x8, xv);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, codes_plus16(word[t]), acc, 0, 0, 0);
          sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, ones, sx, 0, 0, 0);
        }
        // groups wholly beyond K have acc = sx = 0 and a repeated scale
        if (kb * 128 + g * GROUP < a.K)
#pragma unroll
          for (int i = 0; i < 4; ++i) total[i] = fmaf(s, fmaf(-z, sx[i], acc[i]), total[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s_part[wave][q * 4 + i][c] = total[i];
    __syncthreads();
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    if (r0 + tr < n_rows && cb * 16 + tc < a.N) {
      float v = s_part[0][tr][tc];
#pragma unroll
      for (int k = 1; k < kW4Waves; ++k) v += s_part[k][tr][tc];
      st1<ODT>(a.out, (int64_t)s_rows[r0 + tr] * a.N + cb * 16 + tc, v);
    }
    __syncthreads();
  }
}

template <int ODT, int GROUP>
static int launch_group(const GemvW4Args& a, hipStream_t s) {
  const bool by_row = a.experts && a.R < a.E;
  const dim3 grid(a.nb, !a.experts ? 1 : std::min(a.R, a.E));
  if (a.zeros) hipLaunchKernelGGL((gemv_w4_kernel<ODT, GROUP, true>), grid, dim3(kW4Threads), 0, s, a, by_row);
  else hipLaunchKernelGGL((gemv_w4_kernel<ODT, GROUP, false>), grid, dim3(kW4Threads), 0, s, a, by_row);
  return hipGetLastError();
}

template <int ODT>
static int launch_odt(const GemvW4Args& a, hipStream_t s) {
  if (a.group == 32) return launch_group<ODT, 32>(a, s);
  if (a.group == 64) return launch_group<ODT, 64>(a, s);
  return launch_group<ODT, 128>(a, s);
}

int launch_gemv_w4(const GemvW4Args& a, hipStream_t s) {
  return a.out_dt == kBF16 ? launch_odt<kBF16>(a, s) : launch_odt<kF32>(a, s);
}

// The layout: one thread per packed word, then one per scale and zero point.
__global__ __launch_bounds__(kW4Threads) void w4_pack_kernel(W4PackArgs a) {
  const int64_t words = (int64_t)a.E * a.nb * a.kb * 256;
  for (int64_t i = (int64_t)blockIdx.x * kW4Threads + threadIdx.x; i < words; i += (int64_t)gridDim.x * kW4Threads) {
    const int n = (int)(i & 15), q = (int)(i >> 4 & 3), t = (int)(i >> 6 & 3);  // (columns fastest: reads coalesce)
    const int64_t block = i >> 8;                                               // (e * nb + cb) * kb + kb_
    const int kb = (int)(block % a.kb), cb = (int)(block / a.kb % a.nb);
    const int64_t e = block / a.kb / a.nb;
    const int col = cb * 16 + n, k = kb * 128 + t * 32 + q * 8;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t code = col < a.N && k + j < a.K ? a.codes[(e * a.K + k + j) * a.N + col] & 15u : 0u;
      const int at = (3 + 16 * (j & 1) + 4 * (j >> 1)) & 31;
      w |= __builtin_rotateleft32(code, at);
    }
    a.wq[(block * 64 + q * 16 + n) * 4 + t] = w;
  }
  const int64_t scales = (int64_t)a.E * a.nb * a.groups * 16;
  for (int64_t i = (int64_t)blockIdx.x * kW4Threads + threadIdx.x; i < scales; i += (int64_t)gridDim.x * kW4Threads) {
    const int64_t g = i >> 4;
    const int gi = (int)(g % a.groups), cb = (int)(g / a.groups % a.nb);
    const int64_t e = g / a.groups / a.nb;
    const int col = cb * 16 + (int)(i & 15);
    const int64_t from = (e * a.groups + gi) * a.N + col;
    a.scales_out[i] = col < a.N ? a.scales[from] : 0;
    if (a.zeros) a.zeros_out[i] = col < a.N ? a.zeros[from] : 0;
  }
}

int launch_w4_pack(const W4PackArgs& a, hipStream_t s) {
  const int64_t words = (int64_t)a.E * a.nb * a.kb * 256;
  const uint32_t grid = (uint32_t)std::min<int64_t>((words + kW4Threads - 1) / kW4Threads, 16384);
  hipLaunchKernelGGL(w4_pack_kernel, dim3(grid), dim3(kW4Threads), 0, s, a);
  return hipGetLastError();
}

}  // namespace hocf
