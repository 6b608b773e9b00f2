// Products with 8-bit integers, scaled by row and by column.
//
//   out[r][n] = xs[r] ws[e][n] sum_k xq[r][k] wq[e][n][k]
// The sum is exact (32-bit integers), its conversion to fp32 and the two
// factors round once each.  Both operands have their rows' k adjacent, as the
// matrix instruction takes them (16 bytes a lane), so a tile's stages go
// straight from memory to LDS and from there to the instruction.
//
// Bound by the matrix instructions and by what issues beside them: 8192^3 427-439 us (2.5 POP/s,
// where the instruction alone on such numbers reaches 3.95), 8192 x 4096 -> 1792 57-69 us, by the card (224 of 256 CUs
// have a tile; the first loads and the stores are about 12 us of it).
#include "i8_tiles.hpp"
#include "mfma_tile.hpp"
#include "publish.hpp"

namespace hocf {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// A TM x TN tile of four waves; a stage is 128 bytes of k of its rows and columns.  Large tiles
// have two stages and read the next fragments while one's are multiplied.  Small ones, of
// which many share a CU, have four, loaded three steps ahead: their steps are shorter than
// a load takes.
//
// LDS: a row is 128 bytes, eight 16-byte pieces, piece c at c ^ (row / 2 mod 8): 16
// lanes that read one piece of 16 rows touch 16 different groups of banks.
template <int TM_, int TN_>
struct TileI8 {
  static constexpr int TM = TM_, TN = TN_, WM = 2, WN = 2, NW = 4, NT = 256;
  static constexpr int WTM = TM / WM, WTN = TN / WN, FM = WTM / 32, FN = WTN / 32;
  static constexpr int A_BYTES = TM * 128, B_BYTES = TN * 128;
  static constexpr int BK = 128, NST = TM == 64 ? 4 : 2;
  static constexpr int SMEM_BYTES = A_BYTES + B_BYTES;  // one stage
  static constexpr int A_LD = A_BYTES / 1024 / NW, B_LD = B_BYTES / 1024 / NW;

  // acc = rows . columns^T over K (a multiple of 16; rows and columns past the resources' ends
  // and k past K count as zeros).
  __device__ static __forceinline__ void run(__amdgpu_buffer_rsrc_t ra, __amdgpu_buffer_rsrc_t rb, int K,
                                             char* const (&stages)[4], i32x16 (&acc)[FM][FN]) {
    const int lane = opaque_lane(), wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
    // a load instruction fills eight rows: lane l piece l mod 8 of row l / 8; instruction t of a wave
    // is 32 t rows on, which changes neither the piece's place nor the lane's offset
    const int row = wave * 8 + (lane >> 3), piece = ((lane & 7) ^ ((row >> 1) & 7)) << 4;
    const uint32_t off = (uint32_t)row * (uint32_t)K + piece, step32 = 32u * (uint32_t)K;
    auto load_a = [&](char* st, int k0) {
      const uint32_t voff = k0 + piece < K ? off : kNowhere;  // (the last stage may end inside)
#pragma unroll
      for (int t = 0; t < A_LD; ++t) load_lds16(ra, st + (t * NW + wave) * 1024, voff, (uint32_t)k0 + t * step32);
    };
    auto load_b = [&](char* st, int k0) {
      const uint32_t voff = k0 + piece < K ? off : kNowhere;
#pragma unroll
      for (int t = 0; t < B_LD; ++t) load_lds16(rb, st + A_BYTES + (t * NW + wave) * 1024, voff, (uint32_t)k0 + t * step32);
    };
    auto load = [&](char* st, int k0) {
      load_a(st, k0);
      load_b(st, k0);
    };
    // fragment kk of block row i: bytes 32 kk + 16 (lane / 32) of row 32 i + lane mod 32 (blocks are 4 KB
    // apart, kk is two bits of the piece)
    const int m = lane & 31, first = m * BK + (((lane >> 5) ^ ((m >> 1) & 7)) << 4);
    const int afirst = wm * WTM * BK + first, bfirst = A_BYTES + wn * WTN * BK + first;
    auto frags = [&](const char* st, int kk, i32x4 (&a)[FM], i32x4 (&b)[FN]) {
      const char *pa = st + (afirst ^ (kk << 5)), *pb = st + (bfirst ^ (kk << 5));
#pragma unroll
      for (int i = 0; i < FM; ++i) a[i] = *reinterpret_cast<const i32x4*>(pa + i * 32 * BK);
#pragma unroll
      for (int j = 0; j < FN; ++j) b[j] = *reinterpret_cast<const i32x4*>(pb + j * 32 * BK);
    };
    auto mfmas = [&](const i32x4 (&a)[FM], const i32x4 (&b)[FN]) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[j], a[i], acc[i][j], 0, 0, 0);
    };
    constexpr int ND = FM + FN, NM = FM * FN;
    i32x4 a0[FM], b0[FN], a1[FM], b1[FN];
    if constexpr (NST == 4) {
      const int nk = (K + BK - 1) / BK;  // (steps past it load zeros, and cost no memory access)
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        load(stages[s], s * BK);
        in_order();
      }
      auto step = [&](auto s_c, int ks) {
        constexpr int S = decltype(s_c)::value;
        wait_barrier<2 * (A_LD + B_LD)>();  // step ks has arrived, and step ks - 1 is read everywhere
        load(stages[(S + 3) % 4], (ks + 3) * BK);
        in_order();
        frags(stages[S], 0, a0, b0);
        frags(stages[S], 1, a1, b1);
        mfmas(a0, b0);
        frags(stages[S], 2, a0, b0);
        mfmas(a1, b1);
        frags(stages[S], 3, a1, b1);
        mfmas(a0, b0);
        mfmas(a1, b1);
      };
      four_steps(nk, step);
      return;
    }
    // whole pairs of steps: k past K loads as zeros
    const int nk = (K + 2 * BK - 1) / (2 * BK) * 2;
    load(stages[0], 0);
    in_order();
    load_a(stages[1], BK);
    wait_barrier<A_LD>();
    frags(stages[0], 0, a0, b0);
    // Stage S holds step ks.  Its last fragments are read while the third quarter multiplies; the
    // barrier after that frees the stage for step ks + 2 and has step ks + 1 in the other.  Half of a step's
    // loads follow the barrier and half go with the next quarter: in a bunch they hold up the
    // waves that issue them.
    auto step = [&](auto s_c, int ks) {
      constexpr int S = decltype(s_c)::value;
      load_b(stages[S ^ 1], (ks + 1) * BK);
      frags(stages[S], 1, a1, b1);
      mfmas(a0, b0);
      mix<NM, ND, B_LD, 0, 0>();
      frags(stages[S], 2, a0, b0);
      mfmas(a1, b1);
      mix<NM, ND, 0, 0, 0>();
      frags(stages[S], 3, a1, b1);
      mfmas(a0, b0);
      mix<NM, ND, 0, 0, 0>();
      wait_barrier<0>();
      load_a(stages[S], (ks + 2) * BK);
      frags(stages[S ^ 1], 0, a0, b0);
      mfmas(a1, b1);
      mix<NM, ND, A_LD, 0, 0>();
    };
    for (int ks = 0; ks < nk; ks += 2) {
      step(std::integral_constant<int, 0>{}, ks);
      step(std::integral_constant<int, 1>{}, ks + 1);
    }
  }
};

// The matrix kernel: a tile of a group's rows and an expert's columns.
template <class Tile, int ODT>
__global__ __launch_bounds__(256) void gemm_i8_kernel(GemmI8Args a, int ntiles) {
  __shared__ __attribute__((aligned(1024))) char smem0[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem1[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem2[Tile::NST > 2 ? Tile::SMEM_BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char smem3[Tile::NST > 2 ? Tile::SMEM_BYTES : 16];
  char* const stages[4] = {smem0, smem1, smem2, smem3};
  const RowTile t = row_tile<Tile::TM>(a.offsets, a.E, a.T, ntiles, a.sync);
  if (t.e < 0) return;
  const int rows = (int)min((int64_t)Tile::TM, t.end - t.row), col0 = t.nt * Tile::TN, cols = min(Tile::TN, a.N - col0);
  i32x16 acc[Tile::FM][Tile::FN];
  Tile::run(ranged_rsrc(a.xq + t.row * a.K, (uint32_t)rows * (uint32_t)a.K),
            ranged_rsrc(a.wq + ((int64_t)t.e * a.N + col0) * a.K, (uint32_t)cols * (uint32_t)a.K), a.K, stages, acc);
  // lane l, element 4 g + v of block (i, j): row 32 i + l mod 32, column 32 j + 8 g + 4 (l / 32) + v of its wave's part
  const int lane = opaque_lane(), wave = uniform(threadIdx.x >> 6);
  const int r0 = wave / Tile::WN * Tile::WTM + (lane & 31), c0 = wave % Tile::WN * Tile::WTN + 4 * (lane >> 5);
  // (N is a multiple of 8: four columns are all there or none; rows and columns past the tile's end get zeros)
  const __amdgpu_buffer_rsrc_t xs = ranged_rsrc(a.xs + t.row, (uint32_t)rows * 4u);
  const __amdgpu_buffer_rsrc_t ws = ranged_rsrc(a.ws + (int64_t)t.e * a.N + col0, (uint32_t)cols * 4u);
  char* dst = reinterpret_cast<char*>(a.out) + (t.row * a.N + col0) * (ODT == kBF16 ? 2 : 4);
  store_rows<Tile, ODT, false>(
      dst, a.N, rows, cols, stages,
      [&](int i, int j, int g) {
        const float x = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(xs, r0 * 4, 32 * 4 * i, 0));
        const floatx4 w = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(ws, c0 * 4, (32 * j + 8 * g) * 4, 0));
        const i32x16& v = acc[i][j];
        return floatx4{(float)v[4 * g] * x * w[0], (float)v[4 * g + 1] * x * w[1], (float)v[4 * g + 2] * x * w[2],
                       (float)v[4 * g + 3] * x * w[3]};
      },
      [](int, int, floatx4 v) { return v; });
}

template <class Tile, int ODT>
static int launch_tile(const GemmI8Args& a, hipStream_t s) {
  const int ntiles = (a.N + Tile::TN - 1) / Tile::TN;
  hipLaunchKernelGGL((gemm_i8_kernel<Tile, ODT>), row_tile_grid(a.T, a.E, a.offsets, Tile::TM, ntiles), dim3(256), 0, s, a,
                     ntiles);
  return hipGetLastError();
}

template <int ODT>
static int launch_odt(const GemmI8Args& a, hipStream_t s) {
  const int side = tile_side(1, a.T, a.N);
  if (side == 256) return launch_tile<TileI8<256, 256>, ODT>(a, s);
  if (side == 128) return launch_tile<TileI8<128, 128>, ODT>(a, s);
  return launch_tile<TileI8<64, 64>, ODT>(a, s);
}

int launch_gemm_i8(const GemmI8Args& a, hipStream_t s) {
  return a.out_dt == kBF16 ? launch_odt<kBF16>(a, s) : launch_odt<kF32>(a, s);
}

// A few rows, each with an expert of its own choice.  Bound by the weights' bytes.  A
// workgroup takes C blocks of 16 columns of an expert for up to 16 of its rows: its four waves
// take pieces of 128 k in turn (two loads of a lane: 16 columns x 128 bytes, whole lines), U pieces
// at once, and add up in LDS.  Where all of K is at once (C > 1) the rows stay in
// registers and the next block's weights are on their way while one's sums are put together.
// Sums of integers: their order does not matter.
__device__ __forceinline__ int local_expert(const GemvI8Args& a, int r) {
  const uint32_t e = (uint32_t)a.experts[r] - (uint32_t)a.e0;
  return e < (uint32_t)a.E ? (int)e : -1;
}

template <int ODT, int U, int C>
__global__ __launch_bounds__(256) void gemv_i8_kernel(GemvI8Args a, bool by_row) {
  __shared__ int s_part[2][4][16][17];
  __shared__ uint16_t s_rows[kI8MaxRows];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int y = blockIdx.y, n0 = blockIdx.x * 16 * C;
  // this workgroup's expert: the y-th local one, or row y's (and then only for the
  // first of the rows that chose it)
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
    if (mine)
      s_rows[n_rows + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0))] = (uint16_t)r;
    n_rows += __popcll(m);
    // rows of other ranks' experts: zeros, by the row's own workgroup or the first expert's
    if (wave == 0 && a.experts && e < 0 && r < a.R && (by_row ? r == y : y == 0))
      for (int c = n0; c < min(a.N, n0 + 16 * C); ++c) st1<ODT>(a.out, (int64_t)r * a.N + c, 0.0f);
  }
  if (!first || n_rows == 0) return;  // (the same in every wave)
  __builtin_amdgcn_wave_barrier();

  const int q = lane >> 4, c = lane & 15;
  const int8_t* w0 = a.wq + (int64_t)want * a.N * a.K;
  // (columns past the last repeat it, unused; k past K too, as zeros of the rows)
  auto load_w = [&](i32x4 (&w)[U][2], int n, int k0) {
    const int8_t* p = w0 + (int64_t)min(n + c, a.N - 1) * a.K;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[u][h] = *reinterpret_cast<const i32x4*>(p + min(k0 + u * 512 + h * 64 + q * 16, a.K - 16));
  };
  auto load_x = [&](i32x4 (&x)[U][2], int row, int k0) {
    const int8_t* p = a.xq + (int64_t)row * a.K;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) x[u][h] = *reinterpret_cast<const i32x4*>(p + min(k0 + u * 512 + h * 64 + q * 16, a.K - 16));
  };
  auto zero_x = [&](i32x4 (&x)[U][2], int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (k0 + u * 512 + h * 64 + q * 16 >= a.K) x[u][h] = i32x4{0, 0, 0, 0};
  };
  auto products = [&](const i32x4 (&x)[U][2], const i32x4 (&w)[U][2], i32x4 acc) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[u][h], w[u][h], acc, 0, 0, 0);
    return acc;
  };
  for (int r0 = blockIdx.z * 16; r0 < n_rows; r0 += gridDim.z * 16) {
    const int rows = min(16, n_rows - r0);
    const int xrow = s_rows[r0 + min(c, rows - 1)] / a.rows_per_x;
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
    const int r = s_rows[r0 + min(tr, rows - 1)];
    const float xs = a.xs[r / a.rows_per_x];
    // the waves' parts of block n, added up and scaled
    auto fold = [&](const i32x4& acc, int n, int buf) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s_part[buf][wave][q * 4 + i][c] = acc[i];
      lds_barrier();
      if (tr < rows && n + tc < a.N) {
        const int v = s_part[buf][0][tr][tc] + s_part[buf][1][tr][tc] + s_part[buf][2][tr][tc] + s_part[buf][3][tr][tc];
        st1<ODT>(a.out, (int64_t)r * a.N + n + tc, (float)v * xs * a.ws[(int64_t)want * a.N + n + tc]);
      }
    };
    i32x4 xv[U][2], wa[U][2];
    if constexpr (C == 1) {
      i32x4 acc = {0, 0, 0, 0};
      for (int k0 = wave * 128; k0 < a.K; k0 += 512 * U) {
        load_x(xv, xrow, k0);
        load_w(wa, n0, k0);
        zero_x(xv, k0);
        acc = products(xv, wa, acc);
      }
      fold(acc, n0, 0);
      lds_barrier();
    } else {
      const int k0 = wave * 128, end = min(a.N, n0 + 16 * C);
      load_x(xv, xrow, k0);
      load_w(wa, n0, k0);
      zero_x(xv, k0);
      for (int n = n0, buf = 0; n < end; n += 16, buf ^= 1) {
        const i32x4 acc = products(xv, wa, i32x4{0, 0, 0, 0});
        if (n + 16 < end) load_w(wa, n + 16, k0);
        fold(acc, n, buf);
      }
      lds_barrier();
    }
  }
}

template <int ODT, int U, int C>
static int launch_gemv_c(const GemvI8Args& a, int tiles, hipStream_t s) {
  const bool by_row = a.experts && a.R < a.E;
  const dim3 grid((a.N + 16 * C - 1) / (16 * C), !a.experts ? 1 : std::min(a.R, a.E), tiles);
  hipLaunchKernelGGL((gemv_i8_kernel<ODT, U, C>), grid, dim3(256), 0, s, a, by_row);
  return hipGetLastError();
}

template <int ODT, int C>
static int launch_gemv_k(const GemvI8Args& a, int tiles, hipStream_t s) {
  if (a.K <= 512) return launch_gemv_c<ODT, 1, C>(a, tiles, s);
  if (a.K <= 1024) return launch_gemv_c<ODT, 2, C>(a, tiles, s);
  if (a.K <= 2048) return launch_gemv_c<ODT, 4, C>(a, tiles, s);
  return launch_gemv_c<ODT, 8, C>(a, tiles, s);
}

// Blocks of columns a workgroup: as many as leave about 200 workgroups, while all of K is at
// once.  TB/s of weights with 1, 2 and 4 of them: 1 token x 8 of 64 experts 4096 -> 1792 (896 blocks)
// 3.9, 4.4, 4.5; 16 x 2 of 32, 1792 -> 4096 (8192) 4.1, 4.6, 4.8; 16 rows of 4096 x 32768 (2048) 3.6, 4.2,
// 4.6; 8 rows of 1024 x 8192 (512) 2.05, 2.3, 1.6; 1 row of 4096 x 4096 (256) 2.8, 2.4, 1.6.
template <int ODT>
static int launch_gemv(const GemvI8Args& a, hipStream_t s) {
  const int tiles = ((a.R + a.E - 1) / a.E + 15) / 16;
  const int64_t blocks = (int64_t)((a.N + 15) / 16) * (a.experts ? std::min(a.R, a.E) : 1) * tiles;
  if (a.K > 4096 || blocks < 384) return launch_gemv_k<ODT, 1>(a, tiles, s);
  return blocks < 768 ? launch_gemv_k<ODT, 2>(a, tiles, s) : launch_gemv_k<ODT, 4>(a, tiles, s);
}

int launch_gemv_i8(const GemvI8Args& a, hipStream_t s) {
  return a.out_dt == kBF16 ? launch_gemv<kBF16>(a, s) : launch_gemv<kF32>(a, s);
}

}  // namespace hocf
