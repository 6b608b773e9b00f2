// Products of a few token rows with their experts' 4-bit weights.
//
// The weights stream from HBM once; everything else (x, scales) is small.  A
// block of 128 rows x 16 columns is one 16-byte load per lane, laid out as
// the B operand of four 16x16x32 bf16 matrix products (lane q * 16 + n: column
// n, rows 32 t + 8 q + i of word t), with up to 16 token rows as the A
// operand.  A rotation and one mask turn eight codes into the bf16 numbers
// 16 + code; with sx = sum of x over a group (a product with ones),
//   sum x (code - zero) = sum x (16 + code)  -  (16 + zero) sx
// in fp32, then times the group's scale.  That form turns an infinity of x into
// inf - inf, and leaves the range of fp32 from x = 1e37 on: a result that is not
// finite is taken again by the definition, in 64 bits.
//
// A workgroup's four waves take C blocks of 16 columns of an expert together: a
// wave takes every fourth block of rows, and the four fold through LDS in a
// fixed order.  K goes in passes of up to U blocks of a wave (fewer with many
// token rows, whose x is in LDS).  What a wave waits for first is loaded
// first -- x, then scales, then weights, each a straight run of loads, since
// loads come back in order and a load under a condition is waited for at once
// -- so that its products start with the first weights.
//
// Bound by the weights' bytes, and by the 2-3 us until the first of them
// arrive: one token's 8 experts 4096 -> 1792 (30 MB) 8.9 us, 16 tokens x 2 of 32
// experts 1792 -> 4096 (86 MB) 20-22 us.  Beyond 16 rows of an expert, every tile of
// 16 rows reads and decodes its weights again: 4096 x 4096, 16 rows 7.5 us, 32 rows
// 8.8, 64 rows 16, 1024 rows 320.
#include <algorithm>

#include "moe.hpp"
#include "publish.hpp"
#include "sync.hpp"

namespace hocf {

// x in LDS, token rows x rows of W: 16 KB, or 64 KB for more rows than fit
constexpr int kW4X = 8192, kW4XLarge = 32768;
constexpr int kW4Many = 2048;     // (column block, expert) pairs from which a workgroup takes two blocks
constexpr int kW4Few = 512;       // pairs up to which the large x area fits them all at once
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

// One result by the definition (column c of column block `block`, counted over all
// experts).  Slow (K = 4096: 120-140 us in all), and hardly ever needed.
template <int GROUP, bool ZEROS>
__device__ __forceinline__ float by_definition(const GemvW4Args& a, int64_t block, int c, int xrow) {
  const uint16_t* x = a.x + (int64_t)xrow * a.K;
  double sum = 0.0;
#pragma unroll 1
  for (int k = 0; k < a.K; k += 8) {
    const uint32_t w = a.wq[((block * a.kb + k / 128) * 64 + k % 32 / 8 * 16 + c) * 4 + k % 128 / 32];
    const int64_t g = (block * a.groups + k / GROUP) * 16 + c;
    const double s = bf16_to_f32(a.scales[g]), z = ZEROS ? bf16_to_f32(a.zeros[g]) : 8.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t code = __builtin_rotateright32(w, (3 + 16 * (i & 1) + 4 * (i >> 1)) & 31) & 15u;
      sum += (double)bf16_to_f32(x[k + i]) * (s * ((double)code - z));
    }
  }
  return (float)sum;
}

template <int ODT, int GROUP, bool ZEROS, int U, int C, int X>
__global__ __launch_bounds__(256, X > kW4X ? 2 : 4) void gemv_w4_kernel(GemvW4Args a, bool by_row) {
  constexpr int kThreads = 256;
  constexpr int WPG = GROUP / 32;  // words of one group
  constexpr int GPB = 4 / WPG;     // groups of one block
  constexpr int XP = X / 8 / kThreads;  // 16-byte pieces of x that a thread moves
  __shared__ __attribute__((aligned(16))) uint16_t s_x[X + 16 * 8];
  __shared__ float s_part[C][4][16][17];
  __shared__ uint16_t s_rows[kW4MaxRows], s_xrow[kW4MaxRows];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int y = blockIdx.y, cb0 = blockIdx.x * C;
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
      for (int c = cb0 * 16; c < min(a.N, (cb0 + C) * 16); ++c) st1<ODT>(a.out, (int64_t)r * a.N + c, 0.0f);
  }
  if (!first || n_rows == 0) return;  // (the same in every wave)
  __builtin_amdgcn_wave_barrier();

  const int q = lane >> 4, c = lane & 15;
  const int kq = wave;                         // this wave's quarter of K
  const int64_t at0 = (int64_t)want * a.nb;    // (blocks of columns past the last repeat it, unused)
  const Codes codes;
  bool odd = false;  // whether a result of this lane's is not finite
  bf16x8 ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;

  for (int r0 = blockIdx.z * 16; r0 < n_rows; r0 += gridDim.z * 16) {
    const int rows = min(16, n_rows - r0);
    // a pass takes U >> sh blocks of every wave: what fits x's rows
    int sh = 0;
    while (rows > (X / 512 / U) << sh) ++sh;
    const int chunk = (512 * U) >> sh, lp = __builtin_ctz(64 * U) - sh;  // rows of W; log2 of a row of x in pieces
    const int ldx = chunk + 8;                  // (rows of x start on different LDS banks)
    const int row_of = min(c, rows - 1) * ldx;  // (token rows past the last repeat it, unused)
    floatx4 total[C];
#pragma unroll
    for (int n = 0; n < C; ++n) total[n] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < a.K; k0 += chunk) {
      const int blocks = min(chunk, a.kb * 128 - k0) / 128;  // of this pass
      uint4 v[XP];
#pragma unroll
      for (int p = 0; p < XP; ++p) {  // (past the last row or piece: repeated or unused)
        if (p * kThreads >= rows << lp) break;
        const int i = threadIdx.x + p * kThreads, r = min(i >> lp, rows - 1), k = k0 + (i & ((1 << lp) - 1)) * 8;
        v[p] = *reinterpret_cast<const uint4*>(a.x + (int64_t)s_xrow[r0 + r] * a.K + min(k, a.K - 8));
        // rows of W beyond K (in the large area at its store: 16 rows of 4096 x 4096 take 7.8 us with both here)
        if (X == kW4X && k >= a.K) v[p] = make_uint4(0, 0, 0, 0);
      }
      uint4 wv[C][U];
      uint32_t sz[C][U];  // scale and zero
#pragma unroll
      for (int n = 0; n < C; ++n) {
        const int64_t small = (at0 + min(cb0 + n, a.nb - 1)) * a.groups * 16;
        const uint16_t *scales = a.scales + small, *zeros = ZEROS ? a.zeros + small : nullptr;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // lanes of quarter q take the block's group q mod GPB (past the last: repeated, unused)
          const int g0 = (k0 / 128 + min(kq + 4 * u, blocks - 1)) * GPB;
          const uint32_t o = min(q & (GPB - 1), a.groups - 1 - g0) * 16 + c;
          sz[n][u] = scales[g0 * 16 + o];
          if constexpr (ZEROS) sz[n][u] |= (uint32_t)zeros[g0 * 16 + o] << 16;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < C; ++n) {
          const char* wq = reinterpret_cast<const char*>(a.wq) +
                           ((at0 + min(cb0 + n, a.nb - 1)) * a.kb + k0 / 128 + min(kq + 4 * u, blocks - 1)) * 1024;
          wv[n][u] = *reinterpret_cast<const uint4*>(wq + (uint32_t)lane * 16);
        }
      lds_barrier();  // the last pass is done with x
#pragma unroll
      for (int p = 0; p < XP; ++p) {
        if (p * kThreads >= rows << lp) break;
        const int i = threadIdx.x + p * kThreads, r = i >> lp, k = (i & ((1 << lp) - 1)) * 8;
        if (X > kW4X && k0 + k >= a.K) v[p] = make_uint4(0, 0, 0, 0);  // (rows of W beyond K, see above)
        if (r < rows) *reinterpret_cast<uint4*>(&s_x[r * ldx + k]) = v[p];
      }
      lds_barrier();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = kq + 4 * u;
        if (b < blocks) {
#pragma unroll
          for (int g = 0; g < GPB; ++g) {
            floatx4 acc[C], sx = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < C; ++n) acc[n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = g * WPG; t < (g + 1) * WPG; ++t) {
              const bf16x8 xv = *reinterpret_cast<const bf16x8*>(&s_x[row_of + b * 128 + t * 32 + q * 8]);
              sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, ones, sx, 0, 0, 0);
#pragma unroll
              for (int n = 0; n < C; ++n) {
                const uint4& v4 = wv[n][u];
                acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    xv, codes(t == 0 ? v4.x : t == 1 ? v4.y : t == 2 ? v4.z : v4.w), acc[n], 0, 0, 0);
              }
            }
            if (GPB > 1 && k0 + b * 128 + g * GROUP >= a.K) break;  // (groups wholly beyond K have no scale)
#pragma unroll
            for (int n = 0; n < C; ++n) {
              const uint32_t both = GPB == 1 ? sz[n][u] : (uint32_t)__shfl((int)sz[n][u], g * 16 + c, 64);
              const float s = bf16_to_f32(both & 0xffffu);
              const float z = 16.0f + (ZEROS ? __uint_as_float(both & 0xffff0000u) : 8.0f);
#pragma unroll
              for (int i = 0; i < 4; ++i) total[n][i] = fmaf(s, fmaf(-z, sx[i], acc[n][i]), total[n][i]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < C; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_part[n][kq][q * 4 + i][c] = total[n][i];
    lds_barrier();
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
    if (tr < rows) {
      const int64_t out = (int64_t)s_rows[r0 + tr] * a.N;
#pragma unroll
      for (int n = 0; n < C; ++n) {
        const int column = (cb0 + n) * 16 + tc;
        float v = s_part[n][0][tr][tc];
#pragma unroll
        for (int k = 1; k < 4; ++k) v += s_part[n][k][tr][tc];
        if (column < a.N) st1<ODT>(a.out, out + column, v);
        odd |= !(fabsf(v) < INFINITY);
      }
    }
    lds_barrier();
  }
  if (!__any(odd)) return;
  // This lane's results that are not finite (its own stores, read back).  The arguments
  // are read anew: kept until here, they would cost the main loop its registers (5 %).
  auto* args = __builtin_amdgcn_kernarg_segment_ptr();
  __asm__ volatile("" : "+s"(args));
  const GemvW4Args b = *(const GemvW4Args*)args;
  for (int r = blockIdx.z * 16 + (threadIdx.x >> 4); r < n_rows; r += gridDim.z * 16)
    for (int n = 0; n < C; ++n) {
      const int column = (cb0 + n) * 16 + (threadIdx.x & 15);
      const int64_t at = (int64_t)s_rows[r] * b.N + column;
      if (column < b.N && !(fabsf(ld1<ODT>(b.out, at)) < INFINITY))
        st1<ODT>(b.out, at, by_definition<GROUP, ZEROS>(b, at0 + cb0 + n, threadIdx.x & 15, s_xrow[r]));
    }
}

template <int ODT, int GROUP, bool ZEROS, int U, int C, int X>
static int launch_c(const GemvW4Args& a, int tiles, hipStream_t s) {
  const bool by_row = a.experts && a.R < a.E;
  const int y = !a.experts ? 1 : std::min(a.R, a.E);
  hipLaunchKernelGGL((gemv_w4_kernel<ODT, GROUP, ZEROS, U, C, X>), dim3((a.nb + C - 1) / C, y, tiles), dim3(256), 0, s, a,
                     by_row);
  return hipGetLastError();
}

// Few workgroups: one block of columns each, a whole row of blocks in flight.
// Many (more than a device of 256 CUs holds at once): two blocks each, which
// share x, its sums and what a workgroup costs by itself.  Rows are expected
// to spread evenly over the experts: tiles of 16 go to workgroups of their
// own, and more than a tile's share of the small x area takes the large one.
// Measured, the other choice in brackets: two blocks for 4 rows of 4096 x 32768
// (2048 pairs of a column block and an expert) 14.3 us [16.9], one block for 1 row
// of 4096 x 4096 (256 pairs) 4.4 [6.0]; the large area for 8 rows of 4096 x 4096
// 5.9 [7.3] and for 16 rows 7.5 [10.9], the small one for 8 rows of 4096 x 32768
// 15.9 [23.0].
template <int ODT, int GROUP, bool ZEROS>
static int launch_zeros(const GemvW4Args& a, hipStream_t s) {
  const int rows = (a.R + a.E - 1) / a.E, tiles = (rows + 15) / 16;
  const int64_t items = (int64_t)a.nb * std::min(a.R, a.E) * tiles;
  const int u = a.kb <= 8 ? 2 : a.kb <= 16 ? 4 : 8;
  if (std::min(rows, 16) * u * 512 > kW4X && (items <= kW4Few || rows > 8))
    return a.kb <= 8 ? launch_c<ODT, GROUP, ZEROS, 2, 1, kW4XLarge>(a, tiles, s)
                     : launch_c<ODT, GROUP, ZEROS, 4, 1, kW4XLarge>(a, tiles, s);
  if (items >= kW4Many)
    return u == 2 ? launch_c<ODT, GROUP, ZEROS, 2, 2, kW4X>(a, tiles, s) : launch_c<ODT, GROUP, ZEROS, 4, 2, kW4X>(a, tiles, s);
  if (u == 2) return launch_c<ODT, GROUP, ZEROS, 2, 1, kW4X>(a, tiles, s);
  if (u == 4) return launch_c<ODT, GROUP, ZEROS, 4, 1, kW4X>(a, tiles, s);
  return launch_c<ODT, GROUP, ZEROS, 8, 1, kW4X>(a, tiles, s);
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
