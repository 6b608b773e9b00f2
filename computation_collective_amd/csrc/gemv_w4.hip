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
// A workgroup has four waves for each of CB blocks of 16 columns of an expert:
// a wave takes every fourth block of rows, and the four fold through LDS in a
// fixed order.  K goes in passes of up to U blocks of a wave (fewer with many
// token rows, whose x is in LDS).  What a wave waits for first is loaded
// first -- x, then scales, then weights, each a straight run of loads, since
// loads come back in order and a load under a condition is waited for at once
// -- so that its products start with the first weights.
#include <algorithm>

#include "moe.hpp"
#include "publish.hpp"
#include "sync.hpp"

namespace hocf {

constexpr int kW4XElems = 8192;   // x in LDS: token rows x rows of W, 16 KB
constexpr int kW4Pack = 256;      // threads of the packing kernel

// Eight codes of one packed word as 16 + code, in row order: a rotation and one
// and-or per pair.  (The instruction takes no literal: the mask stays in a
// scalar register and the 16s in a vector one, which the compiler would
// otherwise split into two instructions with a literal each.)
struct Codes {
  uint32_t mask = 0x00780078u, sixteens = 0x41804180u;
  __device__ __forceinline__ Codes() {
    __asm__ volatile("" : "+s"(mask));
    __asm__ volatile("" : "+v"(sixteens));
  }
  __device__ __forceinline__ bf16x8 operator()(uint32_t w) const {
    uint4 r;
    r.x = (w & mask) | sixteens;
    r.y = (__builtin_amdgcn_alignbit(w, w, 4) & mask) | sixteens;
    r.z = (__builtin_amdgcn_alignbit(w, w, 8) & mask) | sixteens;
    r.w = (__builtin_amdgcn_alignbit(w, w, 12) & mask) | sixteens;
    return __builtin_bit_cast(bf16x8, r);
  }
};

// Row r's expert among this rank's, or -1.
__device__ __forceinline__ int local_expert(const GemvW4Args& a, int r) {
  const uint32_t e = (uint32_t)a.experts[r] - (uint32_t)a.e0;
  return e < (uint32_t)a.E ? (int)e : -1;
}

template <int ODT, int GROUP, bool ZEROS, int U, int CB>
__global__ __launch_bounds__(256 * CB, 4) void gemv_w4_kernel(GemvW4Args a, bool by_row) {
  constexpr int kThreads = 256 * CB;
  constexpr int WPG = GROUP / 32;  // words of one group
  constexpr int GPB = 4 / WPG;     // groups of one block
  constexpr int XP = kW4XElems / 8 / kThreads;  // 16-byte pieces of x that a thread moves
  __shared__ __attribute__((aligned(16))) uint16_t s_x[kW4XElems + 16 * 8];
  __shared__ float s_part[CB][4][16][17];
  __shared__ uint16_t s_rows[kW4MaxRows], s_xrow[kW4MaxRows];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int y = blockIdx.y, cb0 = blockIdx.x * CB;
  const float per_x = 1.0f / (float)a.rows_per_x;
  // this workgroup's expert: the y-th local one, or row y's (and then only
  // for the first of the rows that chose it)
  const int want = !a.experts ? 0 : by_row ? uniform(local_expert(a, y)) : y;
  int n_rows = 0;
  bool first = true;
  for (int r0 = 0; r0 < a.R; r0 += 64) {
    const int r = r0 + lane;
    const int e = r >= a.R ? -1 : a.experts ? local_expert(a, r) : 0;
    const bool mine = r < a.R && e >= 0 && e == want;
    const uint64_t m = __ballot(mine);
    if (by_row && m && n_rows == 0 && r0 + __builtin_ctzll(m) < y) first = false;
    // (every wave writes the same list: each can use it without waiting for the others)
    if (mine) {
      const int i = n_rows + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
      s_rows[i] = (uint16_t)r;
      s_xrow[i] = (uint16_t)(((float)r + 0.5f) * per_x);  // r / rows_per_x
    }
    n_rows += __popcll(m);
    // rows of other ranks' experts: zeros, by the row's own workgroup or the first expert's
    if (wave == 0 && a.experts && e < 0 && r < a.R && (by_row ? r == y : y == 0))
      for (int c = cb0 * 16; c < min(a.N, (cb0 + CB) * 16); ++c) st1<ODT>(a.out, (int64_t)r * a.N + c, 0.0f);
  }
  if (!first || n_rows == 0) return;  // (the same in every wave)
  __builtin_amdgcn_wave_barrier();

  const int q = lane >> 4, c = lane & 15;
  const int kq = wave & 3, col = wave >> 2;  // this wave's quarter of K, its block of columns
  const int64_t at = (int64_t)want * a.nb + min(cb0 + col, a.nb - 1);  // (past the last block: repeated, unused)
  const char* wq = reinterpret_cast<const char*>(a.wq) + at * a.kb * 1024;
  const uint16_t* scales = a.scales + at * a.groups * 16;
  const uint16_t* zeros = ZEROS ? a.zeros + at * a.groups * 16 : nullptr;
  const Codes codes;
  bf16x8 ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;

  for (int r0 = 0; r0 < n_rows; r0 += 16) {
    const int rows = min(16, n_rows - r0);
    // a pass takes U >> sh blocks of every wave: what fits x's rows
    int sh = 0;
    while (rows > (kW4XElems / 512 / U) << sh) ++sh;
    const int chunk = (512 * U) >> sh, lp = __builtin_ctz(64 * U) - sh;  // rows of W; log2 of a row of x in pieces
    const int ldx = chunk + 8;                  // (rows of x start on different LDS banks)
    const int row_of = min(c, rows - 1) * ldx;  // (token rows past the last repeat it, unused)
    floatx4 total = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < a.K; k0 += chunk) {
      const int blocks = min(chunk, a.kb * 128 - k0) / 128;  // of this pass
      uint4 v[XP];
#pragma unroll
      for (int p = 0; p < XP; ++p) {  // (past the last row or piece: repeated or unused)
        const int i = threadIdx.x + p * kThreads, r = min(i >> lp, rows - 1), k = k0 + (i & ((1 << lp) - 1)) * 8;
        v[p] = *reinterpret_cast<const uint4*>(a.x + (int64_t)s_xrow[r0 + r] * a.K + min(k, a.K - 8));
        if (k >= a.K) v[p] = make_uint4(0, 0, 0, 0);  // rows of W beyond K
      }
      uint4 wv[U];
      uint32_t sz[U], zz[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // lanes of quarter q take the block's group q mod GPB (past the last: repeated, unused)
        const int g0 = (k0 / 128 + min(kq + 4 * u, blocks - 1)) * GPB;
        const uint32_t o = min(q & (GPB - 1), a.groups - 1 - g0) * 16 + c;
        sz[u] = scales[g0 * 16 + o];
        zz[u] = ZEROS ? zeros[g0 * 16 + o] : 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        wv[u] = *reinterpret_cast<const uint4*>(wq + (int64_t)(k0 / 128 + min(kq + 4 * u, blocks - 1)) * 1024 + (uint32_t)lane * 16);
      lds_barrier();  // the last pass is done with x
#pragma unroll
      for (int p = 0; p < XP; ++p) {
        const int i = threadIdx.x + p * kThreads, r = i >> lp;
        if (r < rows) *reinterpret_cast<uint4*>(&s_x[r * ldx + (i & ((1 << lp) - 1)) * 8]) = v[p];
      }
      lds_barrier();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = kq + 4 * u;
        if (b < blocks) {
          const uint32_t word[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
          for (int g = 0; g < GPB; ++g) {
            floatx4 acc = {0.f, 0.f, 0.f, 0.f}, sx = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = g * WPG; t < (g + 1) * WPG; ++t) {
              const bf16x8 xv = *reinterpret_cast<const bf16x8*>(&s_x[row_of + b * 128 + t * 32 + q * 8]);
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, codes(word[t]), acc, 0, 0, 0);
              sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, ones, sx, 0, 0, 0);
            }
            const uint32_t mine = sz[u] | zz[u] << 16;
            const uint32_t both = GPB == 1 ? mine : (uint32_t)__shfl((int)mine, g * 16 + c, 64);
            const float s = bf16_to_f32(both & 0xffffu);
            const float z = 16.0f + (ZEROS ? __uint_as_float(both & 0xffff0000u) : 8.0f);
            if (GPB == 1 || k0 + b * 128 + g * GROUP < a.K)  // (groups wholly beyond K have no scale)
#pragma unroll
              for (int i = 0; i < 4; ++i) total[i] = fmaf(s, fmaf(-z, sx[i], acc[i]), total[i]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s_part[col][kq][q * 4 + i][c] = total[i];
    lds_barrier();
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4 & 15, tb = threadIdx.x >> 8;
    if (tr < rows && (cb0 + tb) * 16 + tc < a.N) {
      float v = s_part[tb][0][tr][tc];
#pragma unroll
      for (int k = 1; k < 4; ++k) v += s_part[tb][k][tr][tc];
      st1<ODT>(a.out, (int64_t)s_rows[r0 + tr] * a.N + (cb0 + tb) * 16 + tc, v);
    }
    if (r0 + 16 < n_rows) lds_barrier();
  }
}

template <int ODT, int GROUP, bool ZEROS, int U>
static int launch_u(const GemvW4Args& a, hipStream_t s) {
  const bool by_row = a.experts && a.R < a.E;
  const int y = !a.experts ? 1 : std::min(a.R, a.E);
  // Many rows of one matrix: four blocks of columns share what a workgroup
  // reads of x, which is then more than it reads of the weights.
  if (!a.experts && a.R > 16)
    hipLaunchKernelGGL((gemv_w4_kernel<ODT, GROUP, ZEROS, 2, 4>), dim3((a.nb + 3) / 4, y), dim3(1024), 0, s, a, by_row);
  else
    hipLaunchKernelGGL((gemv_w4_kernel<ODT, GROUP, ZEROS, U, 1>), dim3(a.nb, y), dim3(256), 0, s, a, by_row);
  return hipGetLastError();
}

template <int ODT, int GROUP, bool ZEROS>
static int launch_zeros(const GemvW4Args& a, hipStream_t s) {
  if (a.kb <= 8) return launch_u<ODT, GROUP, ZEROS, 2>(a, s);
  if (a.kb <= 16) return launch_u<ODT, GROUP, ZEROS, 4>(a, s);
  return launch_u<ODT, GROUP, ZEROS, 8>(a, s);
}

template <int ODT, int GROUP>
static int launch_group(const GemvW4Args& a, hipStream_t s) {
  return a.zeros ? launch_zeros<ODT, GROUP, true>(a, s) : launch_zeros<ODT, GROUP, false>(a, s);
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
__global__ __launch_bounds__(kW4Pack) void w4_pack_kernel(W4PackArgs a) {
  const int64_t words = (int64_t)a.E * a.nb * a.kb * 256;
  for (int64_t i = (int64_t)blockIdx.x * kW4Pack + threadIdx.x; i < words; i += (int64_t)gridDim.x * kW4Pack) {
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
  for (int64_t i = (int64_t)blockIdx.x * kW4Pack + threadIdx.x; i < scales; i += (int64_t)gridDim.x * kW4Pack) {
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
  const uint32_t grid = (uint32_t)std::min<int64_t>((words + kW4Pack - 1) / kW4Pack, 16384);
  hipLaunchKernelGGL(w4_pack_kernel, dim3(grid), dim3(kW4Pack), 0, s, a);
  return hipGetLastError();
}

}  // namespace hocf
