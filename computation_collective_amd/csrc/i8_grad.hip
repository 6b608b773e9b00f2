// Gradients of the 8-bit products, from the codes that the forward pass kept.
//
//   dx[r][k] = sum_n dy[r][n] w[n][k]        w = wq ws rounded to bf16, of r's expert
//   dw[k][n] = sum_r x[r][k] dy[r][n]        x = xq xs rounded to bf16, r over the expert's rows
// and, where the product's rows came through SiLU, dx times its derivative at the
// codes of what SiLU was given.  Codes have no gradient of their own: the rounding
// counts as the identity.
//
// Both sum over the codes' rows, so both read codes alike: a step is 64 rows of
// codes, taken to bf16 on their way through registers to LDS, next to 64 rows
// (dw) or 64 columns (dx) of dy, which go straight to LDS.  Operands whose
// summed index is not adjacent in LDS are turned by the transposing LDS read.
#include "i8_tiles.hpp"

namespace hocf {

// x / (1 + exp(-x)), its derivative.
__device__ __forceinline__ float silu_slope(float h) {
  const float p = 1.0f / (1.0f + __expf(-h));  // (h = -inf: 0, and its slope below NaN, as the formula's)
  return p * fmaf(h, 1.0f - p, 1.0f);
}

// A TR x TC tile (rows x columns of the result) of four waves, summed over steps of 64.
// DW: rows are codes, columns dy, both with the summed index outermost.
// Else: rows are dy with the summed index innermost, columns codes with it outermost.
//
// LDS of an operand with the summed index c outermost: rows of its W numbers, 16-byte pieces
// at piece ^ 4 (c mod 4) (W = 64: ^ 4 (c / 2 mod 2)), so that the transposing read's four rows
// x 64 bytes touch every bank once; innermost: as rows of 128 bytes, piece ^ (row / 2 mod 8).
template <bool DW, int TR, int TC>
struct TileGrad {
  static constexpr int TM = TR, TN = TC, WM = 2, WN = 2, NW = 4, NT = 256;
  static constexpr int WTM = TM / WM, WTN = TN / WN, FM = WTM / 32, FN = WTN / 32;
  static constexpr int BK = 64, NST = 2;
  static constexpr int SMEM_BYTES = (TM + TN) * BK * 2;          // one stage: rows, then columns
  static constexpr int QW = DW ? TR : TC, PW = DW ? TC : TR;     // codes and dy of a step
  static constexpr int Q_AT = DW ? 0 : TM * BK * 2, P_AT = DW ? TM * BK * 2 : 0;
  static constexpr int P_LD = PW * BK * 2 / 1024 / NW;           // 1 KB loads of a wave and step
  static constexpr int QR = 512 / QW, Q_LD = 16 / QR;            // rows of codes of one load; loads of a wave and step
  static_assert(Q_LD >= 1 && P_LD >= 1, "four waves");

  __device__ static __forceinline__ int turn(int W, int c) { return W >= 128 ? 4 * (c & 3) : 4 * ((c >> 1) & 1); }

  struct Operands {
    const uint16_t* dy;  // dx: the tile's first row; dw: the group's first row
    const int8_t* q;     // dx: the expert's codes; dw: the group's first row
    const float* s;      // one scale for each row of q
    int64_t C;           // length of the sum
    int N, K, rows;      // rows: dy's of a dx tile
    int p0, q0;          // dw: first column of dy; first column of q
  };

  __device__ static __forceinline__ void run(const Operands& o, char* const (&stages)[4], floatx16 (&acc)[FM][FN]) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = opaque_lane(), wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    // dy: this lane's part of a 1 KB load
    uint32_t poff;
    int ppiece = 0;
    if constexpr (DW) {
      constexpr int RP = 512 / PW, PC = PW / 8;  // rows of one load; pieces of a row
      const int c = wave * RP + lane / PC;       // (loads are 4 RP rows apart, which does not move the pieces)
      static_assert((NW * RP) % 4 == 0, "pieces stay");
      poff = (uint32_t)c * (uint32_t)o.N * 2u + (uint32_t)(o.p0 * 2) + (((lane % PC) ^ turn(PW, c)) << 4);
    } else {
      const int row = wave * 8 + (lane >> 3);
      ppiece = ((lane & 7) ^ ((row >> 1) & 7)) << 4;
      poff = (uint32_t)row * (uint32_t)o.N * 2u + ppiece;
    }
    const __amdgpu_buffer_rsrc_t rp0 = ranged_rsrc(o.dy, DW ? 0 : (uint32_t)o.rows * (uint32_t)o.N * 2u);
    auto load_p = [&](char* st, int ks) {
      if constexpr (DW) {
        constexpr int RP = 512 / PW;
        const int64_t c0 = (int64_t)ks * BK, left = min((int64_t)BK, max(o.C - c0, (int64_t)0));
        const __amdgpu_buffer_rsrc_t r = ranged_rsrc(o.dy + min(c0, o.C) * o.N, (uint32_t)left * (uint32_t)o.N * 2u);
#pragma unroll
        for (int t = 0; t < P_LD; ++t)
          load_lds16(r, st + P_AT + (t * NW + wave) * 1024, poff, (uint32_t)(t * NW * RP) * (uint32_t)o.N * 2u);
      } else {
        const uint32_t voff = (int64_t)ks * BK * 2 + ppiece < (int64_t)o.N * 2 ? poff : kNowhere;
#pragma unroll
        for (int t = 0; t < P_LD; ++t)
          load_lds16(rp0, st + P_AT + (t * NW + wave) * 1024, voff,
                     (uint32_t)ks * (BK * 2) + (uint32_t)(t * 32) * (uint32_t)o.N * 2u);
      }
    };
    // codes: wave w's rows 16 w .. of a step, QR of them a load, eight codes a lane; and the rows' scales, lane i's row 16 w + i
    const int qrow = lane / (QW / 8), qpiece = lane % (QW / 8);
    const uint32_t qoff = (uint32_t)(wave * 16 + qrow) * (uint32_t)o.K + o.q0 + qpiece * 8;
    struct Codes {
      u32x2 w[Q_LD];
      float s;
    };
    auto load_q = [&](Codes& r, int ks) {
      const int64_t c0 = min((int64_t)ks * BK, o.C);
      const uint32_t left = (uint32_t)min((int64_t)BK, o.C - c0);
      const __amdgpu_buffer_rsrc_t rq = ranged_rsrc(o.q + c0 * o.K, left * (uint32_t)o.K);
#pragma unroll
      for (int t = 0; t < Q_LD; ++t)
        r.w[t] = __builtin_amdgcn_raw_buffer_load_b64(rq, (int)qoff, uniform((int)(t * QR * (uint32_t)o.K)), 0);
      r.s = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ranged_rsrc(o.s + c0, left * 4u),
                                                                           (wave * 16 + (lane & 15)) * 4, 0, 0));
    };
    auto put_q = [&](const Codes& r, char* st, int t) {
      const int c = wave * 16 + t * QR + qrow;
      const float s = __shfl(r.s, t * QR + qrow, 64);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)(r.w[t][i / 4] >> (8 * (i & 3))) * s;
      *reinterpret_cast<u32x4*>(st + Q_AT + c * (QW * 2) + ((qpiece ^ turn(QW, c)) << 4)) =
          u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    };

    typedef short short4v __attribute__((ext_vector_type(4)));
    typedef short short8v __attribute__((ext_vector_type(8)));
    // fragments of quarter kk of a step: summed index innermost
    const int m = lane & 31, inner = (wm * WTM + m) * (BK * 2) + (((lane >> 5) ^ ((m >> 1) & 7)) << 4);
    auto frag_inner = [&](const char* st, int kk, int i) {
      return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(st + (inner ^ (kk << 5)) + i * 32 * BK * 2));
    };
    // outermost: 16 lanes read four rows c x 16 numbers, and lane l gets number l of the four rows
    const int G = lane >> 4, s16 = lane & 15, crow = (G >> 1) * 8 + (s16 >> 2);
    auto outer_at = [&](int W, int w0) {
      const int n = w0 + (G & 1) * 16 + 4 * (s16 & 3);
      return crow * (W * 2) + (((n >> 3) ^ turn(W, crow)) << 4) + (n & 7) * 2;
    };
    auto frag_outer = [&](const char* st, int at, int W, int kk, int j) {
      short4v h[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (HOCF_LDS short4v*)(st + (at ^ (j << 6)) + (kk * 16 + 4 * hh) * (W * 2)));
      return __builtin_bit_cast(bf16x8, short8v{h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]});
    };
    const int rat = outer_at(TM, wm * WTM), cat = outer_at(TN, wn * WTN);
    auto frags = [&](const char* st, int kk, bf16x8 (&a)[FM], bf16x8 (&b)[FN]) {
#pragma unroll
      for (int i = 0; i < FM; ++i) a[i] = DW ? frag_outer(st, rat, TM, kk, i) : frag_inner(st, kk, i);
#pragma unroll
      for (int j = 0; j < FN; ++j) b[j] = frag_outer(st + TM * BK * 2, cat, TN, kk, j);
    };
    auto mfmas = [&](const bf16x8 (&a)[FM], const bf16x8 (&b)[FN]) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
    };
    constexpr int NM = FM * FN, ND = (DW ? 2 : 1) * FM + 2 * FN;
    bf16x8 a0[FM], b0[FN], a1[FM], b1[FN];
    Codes qa, qb;

    // whole pairs of steps: what is past the sum's end loads as zeros
    const int nk = (int)((o.C + 2 * BK - 1) / (2 * BK) * 2);
    if (nk == 0) return;
    load_q(qa, 0);
    load_q(qb, 1);
    in_order();
    load_p(stages[0], 0);
#pragma unroll
    for (int t = 0; t < Q_LD; ++t) put_q(qa, stages[0], t);
    wait_barrier<0>();
    load_p(stages[1], 1);
    in_order();
    load_q(qa, 2);
    frags(stages[0], 0, a0, b0);
    // Stage S holds step ks, whose quarters are multiplied in turn, the next one's fragments on
    // their way; meanwhile step ks + 1's codes become the other stage's numbers.  The barrier before the last quarter
    // has the other stage complete (all but step ks + 2's codes have arrived) and frees stage S,
    // for step ks + 2's dy, and the registers of codes, for step ks + 3's.
    constexpr int T1 = (Q_LD + 2) / 3, T2 = (2 * Q_LD + 2) / 3;
    auto step = [&](auto s_c, int ks, Codes& codes) {
      constexpr int S = decltype(s_c)::value;
      frags(stages[S], 1, a1, b1);
#pragma unroll
      for (int t = 0; t < T1; ++t) put_q(codes, stages[S ^ 1], t);
      mfmas(a0, b0);
      frags(stages[S], 2, a0, b0);
#pragma unroll
      for (int t = T1; t < T2; ++t) put_q(codes, stages[S ^ 1], t);
      mfmas(a1, b1);
      frags(stages[S], 3, a1, b1);
#pragma unroll
      for (int t = T2; t < Q_LD; ++t) put_q(codes, stages[S ^ 1], t);
      mfmas(a0, b0);
      wait_barrier<Q_LD + 1>();
      load_p(stages[S], ks + 2);
      in_order();
      load_q(codes, ks + 3);
      frags(stages[S ^ 1], 0, a0, b0);
      mfmas(a1, b1);
    };
    for (int ks = 0; ks < nk; ks += 2) {
      step(std::integral_constant<int, 0>{}, ks, qb);
      step(std::integral_constant<int, 1>{}, ks + 1, qa);
    }
#endif
  }
};

template <class Tile, int ODT, bool SILU>
__global__ __launch_bounds__(256) void gemm_i8_dx_kernel(GradI8Args a, int ntiles) {
  __shared__ __attribute__((aligned(1024))) char smem0[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem1[Tile::SMEM_BYTES];
  char* const stages[4] = {smem0, smem1, smem0, smem1};
  const RowTile t = row_tile<Tile::TM>(a.offsets, a.E, a.T, ntiles, a.sync);
  if (t.e < 0) return;
  const int rows = (int)min((int64_t)Tile::TM, t.end - t.row), col0 = t.nt * Tile::TN, cols = min(Tile::TN, a.K - col0);
  floatx16 acc[Tile::FM][Tile::FN];
  Tile::run({a.dy + t.row * a.N, a.q + (int64_t)t.e * a.N * a.K, a.s + (int64_t)t.e * a.N, a.N, a.N, a.K, rows, 0, col0},
            stages, acc);
  char* dst = reinterpret_cast<char*>(a.out) + (t.row * a.K + col0) * (ODT == kBF16 ? 2 : 4);
  const int8_t* pre = SILU ? a.pre + t.row * a.K + col0 : nullptr;
  const float* pre_s = SILU ? a.pre_s + t.row : nullptr;
  store_rows<Tile, ODT, SILU>(
      dst, a.K, rows, cols, stages,
      [&](int i, int j, int g) {
        const floatx16& v = acc[i][j];
        return floatx4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
      },
      [&](int r, int c, floatx4 v) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(pre + (int64_t)r * a.K + c);
        const float s = pre_s[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= silu_slope(bf16_to_f32(f32_to_bf16((float)(int8_t)(q >> (8 * i)) * s)));
        return v;
      });
}

template <class Tile, int ODT>
__global__ __launch_bounds__(256) void gemm_i8_dw_kernel(GradI8Args a, int ktiles, int ntiles) {
  __shared__ __attribute__((aligned(1024))) char smem0[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem1[Tile::SMEM_BYTES];
  char* const stages[4] = {smem0, smem1, smem0, smem1};
  // each XCD takes one run of all tiles, expert by expert, row tile by row tile
  const int64_t total = (int64_t)a.E * ktiles * ntiles, b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int q = (int)(b % kNumQueues);
  const int64_t at = total * q / kNumQueues + b / kNumQueues;
  if (at >= total * (q + 1) / kNumQueues) return;
  const int e = (int)(at / ((int64_t)ktiles * ntiles)), in = (int)(at - (int64_t)e * ktiles * ntiles);
  const int k0 = in / ntiles * Tile::TM, n0 = in % ntiles * Tile::TN;
  int64_t lo = 0, hi = a.T;
  if (a.offsets) {
    group_bounds(a.offsets, e, a.T, &lo, &hi);
    if (in == 0 && threadIdx.x == 0 && (lo != a.offsets[e] || hi != a.offsets[e + 1])) report_status(a.sync, kErrBadIndex);
    lo = uniform64(lo);
    hi = uniform64(hi);
  }
  floatx16 acc[Tile::FM][Tile::FN];
  Tile::run({a.dy + lo * a.N, a.q + lo * a.K, a.s + lo, hi - lo, a.N, a.K, 0, n0, k0}, stages, acc);
  char* dst = reinterpret_cast<char*>(a.out) + (((int64_t)e * a.K + k0) * a.N + n0) * (ODT == kBF16 ? 2 : 4);
  store_rows<Tile, ODT, false>(
      dst, a.N, min(Tile::TM, a.K - k0), min(Tile::TN, a.N - n0), stages,
      [&](int i, int j, int g) {
        const floatx16& v = acc[i][j];
        return floatx4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
      },
      [](int, int, floatx4 v) { return v; });
}

template <class Tile, int ODT>
static int launch_dx_tile(const GradI8Args& a, hipStream_t s) {
  const int ntiles = (a.K + Tile::TN - 1) / Tile::TN;
  const dim3 grid = row_tile_grid(a.T, a.E, a.offsets, Tile::TM, ntiles);
  if (a.pre) hipLaunchKernelGGL((gemm_i8_dx_kernel<Tile, ODT, true>), grid, dim3(256), 0, s, a, ntiles);
  else hipLaunchKernelGGL((gemm_i8_dx_kernel<Tile, ODT, false>), grid, dim3(256), 0, s, a, ntiles);
  return hipGetLastError();
}
template <int ODT>
static int launch_dx(const GradI8Args& a, hipStream_t s) {
  const int64_t big = ((a.T + 255) / 256) * ((a.K + 255) / 256), mid = ((a.T + 127) / 128) * ((a.K + 127) / 128);
  if (big >= 128) return launch_dx_tile<TileGrad<false, 256, 256>, ODT>(a, s);
  if (mid >= 128) return launch_dx_tile<TileGrad<false, 128, 128>, ODT>(a, s);
  return launch_dx_tile<TileGrad<false, 64, 64>, ODT>(a, s);
}
int launch_gemm_i8_dx(const GradI8Args& a, hipStream_t s) {
  return a.out_dt == kBF16 ? launch_dx<kBF16>(a, s) : launch_dx<kF32>(a, s);
}

template <class Tile, int ODT>
static int launch_dw_tile(const GradI8Args& a, hipStream_t s) {
  const int kt = (a.K + Tile::TM - 1) / Tile::TM, nt = (a.N + Tile::TN - 1) / Tile::TN;
  const int64_t n = ((int64_t)a.E * kt * nt + kNumQueues - 1) / kNumQueues * kNumQueues, x = std::min<int64_t>(n, 1 << 20);
  hipLaunchKernelGGL((gemm_i8_dw_kernel<Tile, ODT>), dim3((uint32_t)x, (uint32_t)((n + x - 1) / x)), dim3(256), 0, s, a, kt, nt);
  return hipGetLastError();
}
template <int ODT>
static int launch_dw(const GradI8Args& a, hipStream_t s) {
  const int64_t big = (int64_t)a.E * ((a.K + 255) / 256) * ((a.N + 255) / 256);
  const int64_t mid = (int64_t)a.E * ((a.K + 127) / 128) * ((a.N + 127) / 128);
  if (big >= 128) return launch_dw_tile<TileGrad<true, 256, 256>, ODT>(a, s);
  if (mid >= 128) return launch_dw_tile<TileGrad<true, 128, 128>, ODT>(a, s);
  return launch_dw_tile<TileGrad<true, 64, 64>, ODT>(a, s);
}
int launch_gemm_i8_dw(const GradI8Args& a, hipStream_t s) {
  return a.out_dt == kBF16 ? launch_dw<kBF16>(a, s) : launch_dw<kF32>(a, s);
}

}  // namespace hocf
