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
//
// Bound by the matrix instructions and by what issues beside them: of a step's 3340 cycles (256 x
// 256, dx) 2048 multiply, some 300 go to LDS reads, conversions and barriers, and about 50 to each of the
// 18 loads, for which a wave holds its matrix pipe.  8192 rows, 4096 -> 1792: dx 114-127 us, through SiLU 25 more, dw (fp32)
// 130-144 as one matrix in two parts (one card and another).
#include "i8_tiles.hpp"

namespace hocf {

// The derivative of x / (1 + exp(-x)) at a bf16 number h: p (1 + h (1 - p)), p = 1 / (1 + exp(-h)).  With z =
// exp(-|h|), p and 1 - p are 1 / (1 + z) and z / (1 + z), or the other way round: neither is a difference.  h
// times the first 16 bits of log2(e) is exact, so the exponential's error does not grow with h; the rest of
// log2(e) is the factor exp(-|h| rest) = 1 - |h| rest, off by 2^-23 at most where z is not zero (below |h| = 88).
__device__ __forceinline__ float silu_slope(float h) {
  constexpr double kHead = 47274.0 / 32768, kRest = (1.4426950408889634 - kHead) * 0.6931471805599453;
  float z = __builtin_amdgcn_exp2f(fabsf(h) * (float)-kHead);
  z = fmaf(z, fabsf(h) * (float)-kRest, z);
  const float i = __builtin_amdgcn_rcpf(1.0f + z), zi = z * i;
  return (h < 0.0f ? zi : i) * fmaf(h, h < 0.0f ? i : zi, 1.0f);
}

// A TR x TC tile (rows x columns of the result) of four waves, summed over steps of 64.
// DW: rows are codes, columns dy.  Else: rows are dy, columns codes.
//
// LDS: a row is one row or column of the tile, 128 bytes of the summed index c in eight
// 16-byte pieces.  dx's dy comes like that, piece p at p ^ (row / 2 mod 8).  Codes have c
// outermost in memory: a thread takes a block of 8 c x 8 columns, whose numbers
// it turns on their way (piece p of column n at p ^ (n / 2 mod 8) ^ (n / 8 mod 8): the writes
// of eight columns apart and the reads of neighbours both touch every bank once).  dw's dy
// has c outermost too and goes straight to LDS as it is, rows of c, pieces at p ^ 4 (c mod 4)
// (64 columns: ^ 4 (c / 2 mod 2)); the transposing read turns it, four rows x 64 bytes at a time.
//
// Small tiles have few steps' work between barriers: two groups of four waves each sum half of the
// steps, and the first adds the second's.
template <bool DW, int TR, int TC>
struct TileGrad {
  static constexpr int TM = TR, TN = TC, WM = 2, WN = 2, NW = 4, NT = 256, GROUPS = TR == 64 ? 2 : 1;
  static constexpr int WTM = TM / WM, WTN = TN / WN, FM = WTM / 32, FN = WTN / 32;
  // Two stages of dy and of codes (which wait in registers before), each an array of its own:
  // the compiler then knows that what is on its way into one is not read or written in another.
  static constexpr int BK = 64, NST = 4;
  static constexpr int QW = DW ? TR : TC, PW = DW ? TC : TR;     // codes and dy of a step
  static constexpr int SMEM_BYTES = TM * BK * 2;
  static_assert(TM == TN, "arrays of one size");
  static constexpr int P_LD = PW * BK * 2 / 1024 / NW;           // 1 KB loads of a wave and step
  static constexpr int QR = QW == 64 ? 4 : 8, QC = QW * BK / NT / QR;  // a thread's block of codes
  static constexpr int Q_LD = QR + QR / 4;                       // its loads: rows of codes, and their scales
  static_assert((QC == 8 || QC == 4) && P_LD >= 1, "four waves");

  struct Operands {
    const uint16_t* dy;  // dx: the tile's first row; dw: the group's first row
    const int8_t* q;     // dx: the expert's codes; dw: the group's first row
    const float* s;      // one scale for each row of q
    int64_t C;           // length of the sum
    int N, K, rows;      // rows: dy's of a dx tile
    int p0, q0;          // dw: first column of dy; first column of q
    // its half of the steps, `n` each
    __device__ __forceinline__ Operands half(int group, int n) const {
      const int64_t first = min((int64_t)n * BK, C), from = group ? first : 0;
      return {dy + from * (DW ? N : 1), q + from * K, s + from, group ? C - first : first, N, K, rows, p0, q0};
    }
  };
  // Steps of a sum, in whole pairs, of one group.
  __device__ static __forceinline__ int steps(int64_t C) {
    return (int)((C + 2 * GROUPS * BK - 1) / (2 * GROUPS * BK) * 2);
  }

  // All of a workgroup's sum, in the first group's accumulators.
  __device__ static __forceinline__ void sum(const Operands& o, char* const (&st)[8], floatx16 (&acc)[FM][FN]) {
    const int n = steps(o.C);
    if constexpr (GROUPS == 1) {
      run(o, n, {st[0], st[1]}, {st[2], st[3]}, acc);
    } else {
      const int group = uniform(threadIdx.x >> 8);
      if (group == 0) run(o.half(0, n), n, {st[0], st[1]}, {st[2], st[3]}, acc);
      else run(o.half(1, n), n, {st[4], st[5]}, {st[6], st[7]}, acc);
      wait_barrier<0>();
      static_assert(FM == 1 && FN == 1 && SMEM_BYTES == 8 * NT * 4, "the second group's accumulators in two of its arrays");
      if (group) {
#pragma unroll
        for (int v = 0; v < 16; ++v) reinterpret_cast<float*>(st[4 + v / 8])[v % 8 * NT + threadIdx.x % NT] = acc[0][0][v];
      }
      wait_barrier<0>();
      if (!group) {
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[0][0][v] += reinterpret_cast<const float*>(st[4 + v / 8])[v % 8 * NT + threadIdx.x];
      }
    }
  }

  struct Two {
    char* at[2];
    __device__ __forceinline__ char* operator[](int i) const { return at[i]; }
  };
  // nk steps (even; the same in both groups, whose barriers they share)
  __device__ static __forceinline__ void run(const Operands& o, int nk, const Two& ps, const Two& qs, floatx16 (&acc)[FM][FN]) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = opaque_lane(), wave = uniform((threadIdx.x >> 6) % NW);
    const int wm = wave / WN, wn = wave % WN;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    // dy: this lane's part of a 1 KB load
    constexpr int RP = 512 / PW, PC = PW / 8;  // dw: rows of one load; pieces of a row
    auto turn = [](int c) { return PW >= 128 ? 4 * (c & 3) : 4 * ((c >> 1) & 1); };
    uint32_t poff;
    int ppiece = 0;
    if constexpr (DW) {
      const int c = wave * RP + lane / PC;     // (loads are 4 RP rows apart, which does not move the pieces)
      static_assert((NW * RP) % 4 == 0, "pieces stay");
      poff = (uint32_t)c * (uint32_t)o.N * 2u + (uint32_t)(o.p0 * 2) + (((lane % PC) ^ turn(c)) << 4);
    } else {
      const int row = wave * 8 + (lane >> 3);
      ppiece = ((lane & 7) ^ ((row >> 1) & 7)) << 4;
      poff = (uint32_t)row * (uint32_t)o.N * 2u + ppiece;
    }
    // (dx: o.C columns of dy's rows from here; the last row ends o.N - o.C columns early, or more)
    const __amdgpu_buffer_rsrc_t rp0 =
        ranged_rsrc(o.dy, DW ? 0 : ((uint32_t)(o.rows - 1) * (uint32_t)o.N + (uint32_t)o.C) * 2u);
    auto load_p = [&](char* st, int ks, int t0, int t1) {
      if constexpr (DW) {
        const int64_t c0 = min((int64_t)ks * BK, o.C);
        const uint32_t left = (uint32_t)min((int64_t)BK, o.C - c0);
        const __amdgpu_buffer_rsrc_t r = ranged_rsrc(o.dy + c0 * o.N, left * (uint32_t)o.N * 2u);
#pragma unroll
        for (int t = t0; t < t1; ++t)
          load_lds16(r, st + (t * NW + wave) * 1024, poff, (uint32_t)(t * NW * RP) * (uint32_t)o.N * 2u);
      } else {
        const uint32_t voff = (int64_t)ks * BK * 2 + ppiece < o.C * 2 ? poff : kNowhere;
#pragma unroll
        for (int t = t0; t < t1; ++t)
          load_lds16(rp0, st + (t * NW + wave) * 1024, voff,
                     (uint32_t)ks * (BK * 2) + (uint32_t)(t * 32) * (uint32_t)o.N * 2u);
      }
    };
    // codes: QR rows x QC columns a thread, and the rows' scales
    const int tid = wave * 64 + lane, qcol = tid % (QW / QC) * QC, qrow = tid / (QW / QC) * QR;
    const uint32_t qoff = (uint32_t)qrow * (uint32_t)o.K + (uint32_t)(o.q0 + qcol);
    struct Codes {
      uint32_t w[QR][QC / 4];
      floatx4 s[QR / 4];
    };
    auto load_q = [&](Codes& r, int ks, int l0, int l1) {
      const int64_t c0 = min((int64_t)ks * BK, o.C);
      const uint32_t left = (uint32_t)min((int64_t)BK, o.C - c0);
      const __amdgpu_buffer_rsrc_t rq = ranged_rsrc(o.q + c0 * o.K, left * (uint32_t)o.K), rs = ranged_rsrc(o.s + c0, left * 4u);
#pragma unroll
      for (int l = l0; l < l1; ++l) {
        if (l < QR / 4) {
          r.s[l] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(rs, qrow * 4 + l * 16, 0, 0));
          continue;
        }
        const int t = l - QR / 4, soff = uniform((int)(t * (uint32_t)o.K));
        if constexpr (QC == 8) {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rq, (int)qoff, soff, 0);
          r.w[t][0] = v[0];
          r.w[t][QC / 4 - 1] = v[1];
        } else {
          r.w[t][0] = __builtin_amdgcn_raw_buffer_load_b32(rq, (int)qoff, soff, 0);
        }
      }
    };
    // column i of the block
    const int qpiece = qrow >> 3, qhalf = (qrow & 4) * 2;
    auto put_q = [&](const Codes& r, char* st, int i) {
      const int n = qcol + i;
      float v[QR];
#pragma unroll
      for (int t = 0; t < QR; ++t) v[t] = (float)(int8_t)(r.w[t][i / 4] >> (8 * (i & 3))) * r.s[t / 4][t & 3];
      char* p = st + n * (BK * 2) + ((qpiece ^ ((n >> 1) & 7) ^ ((n >> 3) & 7)) << 4) + qhalf;
      if constexpr (QR == 8)
        *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[QR - 4], v[QR - 3]),
                                             pack_bf16x2(v[QR - 2], v[QR - 1])};
      else
        *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };

    typedef short short4v __attribute__((ext_vector_type(4)));
    typedef short short8v __attribute__((ext_vector_type(8)));
    // fragments of quarter kk of a step: pieces 2 kk + lane / 32 of rows lane mod 32 of each block
    const int m = lane & 31, half = lane >> 5;
    const int p_at = (wm * WTM + m) * (BK * 2) + ((half ^ ((m >> 1) & 7)) << 4);                // (dx)
    const int qw0 = (DW ? wm * WTM : wn * WTN) + m;
    const int q_at = qw0 * (BK * 2) + ((half ^ ((qw0 >> 1) & 7) ^ ((qw0 >> 3) & 7)) << 4);
    auto frag_p = [&](const char* st, int kk, int i) {
      return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(st + (p_at ^ (kk << 5)) + i * 32 * BK * 2));
    };
    auto frag_q = [&](const char* st, int kk, int i) {  // (32 columns on: n / 8 mod 8 changes by 4)
      return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(st + (q_at ^ (kk << 5) ^ ((i & 1) << 6)) + i * 32 * BK * 2));
    };
    // dw's dy: 16 lanes read four rows c x 16 numbers, and lane l gets number l of the four rows
    const int G = lane >> 4, s16 = lane & 15, crow = (G >> 1) * 8 + (s16 >> 2), pn = wn * WTN + (G & 1) * 16 + 4 * (s16 & 3);
    const int t_at = crow * (PW * 2) + (((pn >> 3) ^ turn(crow)) << 4) + (pn & 7) * 2;
    auto frag_t = [&](const char* st, int kk, int j) {
      short4v h[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (HOCF_LDS short4v*)(st + (t_at ^ (j << 6)) + (kk * 16 + 4 * hh) * (PW * 2)));
      return __builtin_bit_cast(bf16x8, short8v{h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]});
    };
    auto frags = [&](const char* p, const char* q, int kk, bf16x8 (&a)[FM], bf16x8 (&b)[FN]) {
#pragma unroll
      for (int i = 0; i < FM; ++i) a[i] = DW ? frag_q(q, kk, i) : frag_p(p, kk, i);
#pragma unroll
      for (int j = 0; j < FN; ++j) b[j] = DW ? frag_t(p, kk, j) : frag_q(q, kk, j);
    };
    auto mfmas = [&](const bf16x8 (&a)[FM], const bf16x8 (&b)[FN]) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
    };
    constexpr int NM = FM * FN, ND = FM + (DW ? 2 : 1) * FN;
    bf16x8 a0[FM], b0[FN], a1[FM], b1[FN];
    Codes qa, qb;
    // (what is past the sum's end loads as zeros)
    if (nk == 0) return;
    // a step's loads: dy's in two runs, the codes' in three (the last quarter's before the first two of the next step)
    constexpr int P0 = P_LD / 2, Q0 = Q_LD / 3, Q1 = 2 * Q_LD / 3;
    load_q(qa, 0, 0, Q_LD);
    load_p(ps[0], 0, 0, P_LD);
    in_order();
    load_q(qb, 1, 0, Q_LD);
#pragma unroll
    for (int i = 0; i < QC; ++i) put_q(qa, qs[0], i);
    wait_barrier<Q_LD>();
    load_p(ps[1], 1, 0, P0);
    load_q(qa, 2, 0, Q0);
    frags(ps[0], qs[0], 0, a0, b0);
    in_order();
    // Step ks multiplies its quarters in turn, the next one's fragments on their way; meanwhile the codes of
    // step ks + 1 become numbers in the other stage.  At the barrier before the last quarter that stage is complete
    // (of the loads, only those behind its dy may still be on their way), and what step ks read is free: for step ks + 2's dy,
    // and the registers of codes for step ks + 3's.  Their loads are spread over three quarters:
    // in a bunch they hold up the waves that issue them.
    constexpr int C1 = (QC + 2) / 3, C2 = (2 * QC + 2) / 3, VC = QR * 5 / 2;  // (vector instructions of a column)
    auto step = [&](auto s_c, int ks, Codes& next, Codes& after) {
      constexpr int S = decltype(s_c)::value;
      load_p(ps[S ^ 1], ks + 1, P0, P_LD);
      in_order();
      load_q(after, ks + 2, Q0, Q1);
      frags(ps[S], qs[S], 1, a1, b1);
#pragma unroll
      for (int i = 0; i < C1; ++i) put_q(next, qs[S ^ 1], i);
      mfmas(a0, b0);
      mix<NM, ND, P_LD - P0 + Q1 - Q0, C1 * VC, C1>();
      load_q(after, ks + 2, Q1, Q_LD);
      frags(ps[S], qs[S], 2, a0, b0);
#pragma unroll
      for (int i = C1; i < C2; ++i) put_q(next, qs[S ^ 1], i);
      mfmas(a1, b1);
      mix<NM, ND, Q_LD - Q1, (C2 - C1) * VC, C2 - C1>();
      frags(ps[S], qs[S], 3, a1, b1);
#pragma unroll
      for (int i = C2; i < QC; ++i) put_q(next, qs[S ^ 1], i);
      mfmas(a0, b0);
      mix<NM, ND, 0, (QC - C2) * VC, QC - C2>();
      wait_barrier<Q_LD - Q0>();
      load_p(ps[S], ks + 2, 0, P0);
      load_q(next, ks + 3, 0, Q0);
      frags(ps[S ^ 1], qs[S ^ 1], 0, a0, b0);
      mfmas(a1, b1);
      mix<NM, ND, P0 + Q0, 0, 0>();
    };
    for (int ks = 0; ks < nk; ks += 2) {
      step(std::integral_constant<int, 0>{}, ks, qb, qa);
      step(std::integral_constant<int, 1>{}, ks + 1, qa, qb);
    }
#endif
  }
};

template <class Tile, int ODT, bool SILU>
__global__ __launch_bounds__(256 * Tile::GROUPS) void gemm_i8_dx_kernel(GradI8Args a, int ntiles) {
  __shared__ __attribute__((aligned(1024))) char smem0[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem1[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem2[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem3[Tile::SMEM_BYTES];
  constexpr int kSecond = Tile::GROUPS == 2 ? Tile::SMEM_BYTES : 16;
  __shared__ __attribute__((aligned(1024))) char smem4[kSecond];
  __shared__ __attribute__((aligned(1024))) char smem5[kSecond];
  __shared__ __attribute__((aligned(1024))) char smem6[kSecond];
  __shared__ __attribute__((aligned(1024))) char smem7[kSecond];
  char* const stages[4] = {smem0, smem1, smem2, smem3};
  char* const all[8] = {smem0, smem1, smem2, smem3, smem4, smem5, smem6, smem7};
  const RowTile t = row_tile<Tile::TM>(a.offsets, a.E, a.T, ntiles, a.sync);
  if (t.e < 0) return;
  const int rows = (int)min((int64_t)Tile::TM, t.end - t.row), col0 = t.nt * Tile::TN, cols = min(Tile::TN, a.K - col0);
  floatx16 acc[Tile::FM][Tile::FN];
  Tile::sum({a.dy + t.row * a.N, a.q + (int64_t)t.e * a.N * a.K, a.s + (int64_t)t.e * a.N, a.N, a.N, a.K, rows, 0, col0},
            all, acc);
  if (Tile::GROUPS > 1 && threadIdx.x >= 256) {
    wait_barrier<0>();  // (store_rows')
    return;
  }
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

// The expert of rank r when experts stand by falling rows (up to 64; by number where there are more, and among equals).
__device__ __forceinline__ int expert_of_rank(const GradI8Args& a, int r) {
  if (a.E > 64 || !a.offsets) return r;
  const int lane = threadIdx.x & 63;
  int lo, hi, upto = 0;
  lane_bounds(a.offsets, a.E, a.T, 0, false, &upto, &lo, &hi);  // (where they fall: any order, the same for all)
  const int n = lane < a.E ? hi - lo : -1;
  int before = 0;
  for (int i = 0; i < a.E; ++i) {
    const int o = __shfl(n, i, 64);
    before += o > n || (o == n && i < lane);
  }
  return __builtin_ctzll(__ballot(lane < a.E && before == r));
}

// A tile of an expert's matrix, or of one of `splits` parts of the sum over its rows (then in
// fp32 to the workspace, which holds the parts one after another).  Every XCD takes an eighth of
// each expert's tiles, the experts with most rows first: groups differ in length, and what is
// long is not to be left for the end (three groups of 8192 rows in all, 112 tiles each: on average
// 73 steps of 64 rows a CU, 119 with the experts' tiles dealt to the XCDs as they stand, 57 at best).
template <class Tile, int ODT>
__global__ __launch_bounds__(256 * Tile::GROUPS) void gemm_i8_dw_kernel(GradI8Args a, int ktiles, int ntiles, int splits) {
  __shared__ __attribute__((aligned(1024))) char smem0[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem1[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem2[Tile::SMEM_BYTES];
  __shared__ __attribute__((aligned(1024))) char smem3[Tile::SMEM_BYTES];
  constexpr int kSecond = Tile::GROUPS == 2 ? Tile::SMEM_BYTES : 16;
  __shared__ __attribute__((aligned(1024))) char smem4[kSecond];
  __shared__ __attribute__((aligned(1024))) char smem5[kSecond];
  __shared__ __attribute__((aligned(1024))) char smem6[kSecond];
  __shared__ __attribute__((aligned(1024))) char smem7[kSecond];
  char* const stages[4] = {smem0, smem1, smem2, smem3};
  char* const all[8] = {smem0, smem1, smem2, smem3, smem4, smem5, smem6, smem7};
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, i = b / kNumQueues;
  const int q = (int)(b % kNumQueues), units = ktiles * ntiles * splits;
  const int most = (units + kNumQueues - 1) / kNumQueues;  // of one expert on one XCD
  const int rank = (int)(i / most);
  const int unit = (int)((int64_t)units * q / kNumQueues + i % most);
  if (rank >= a.E || unit >= (int)((int64_t)units * (q + 1) / kNumQueues)) return;
  const int e = uniform(expert_of_rank(a, rank)), part = unit / (ktiles * ntiles), in = unit - part * (ktiles * ntiles);
  const int k0 = in / ntiles * Tile::TM, n0 = in % ntiles * Tile::TN;
  int64_t lo = 0, hi = a.T;
  if (a.offsets) {
    group_bounds(a.offsets, e, a.T, &lo, &hi);
    if (in == 0 && threadIdx.x == 0 && (lo != a.offsets[e] || hi != a.offsets[e + 1])) report_status(a.sync, kErrBadIndex);
  }
  if (splits > 1) {
    const int64_t steps = (hi - lo + Tile::BK - 1) / Tile::BK, first = lo;
    lo = min(first + steps * part / splits * Tile::BK, hi);
    hi = min(first + steps * (part + 1) / splits * Tile::BK, hi);
  }
  floatx16 acc[Tile::FM][Tile::FN];
  Tile::sum({a.dy + lo * a.N, a.q + lo * a.K, a.s + lo, hi - lo, a.N, a.K, 0, n0, k0}, all, acc);
  if (Tile::GROUPS > 1 && threadIdx.x >= 256) {
    wait_barrier<0>();  // (store_rows')
    return;
  }
  char* dst = reinterpret_cast<char*>(a.out) + ((((int64_t)part * a.E + e) * a.K + k0) * a.N + n0) * (ODT == kBF16 ? 2 : 4);
  store_rows<Tile, ODT, false>(
      dst, a.N, min(Tile::TM, a.K - k0), min(Tile::TN, a.N - n0), stages,
      [&](int i, int j, int g) {
        const floatx16& v = acc[i][j];
        return floatx4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
      },
      [](int, int, floatx4 v) { return v; });
}

// The parts of the sums, added in order.
template <int ODT>
__global__ __launch_bounds__(256) void dw_sum_kernel(const float* part, void* out, int64_t n, int splits) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
    floatx4 v = *reinterpret_cast<const floatx4*>(part + i);
    for (int c = 1; c < splits; ++c) v = v + *reinterpret_cast<const floatx4*>(part + c * n + i);
    st4<ODT>(out, i, v);
  }
}

template <class Tile, int ODT>
static int launch_dx_tile(const GradI8Args& a, hipStream_t s) {
  const int ntiles = (a.K + Tile::TN - 1) / Tile::TN;
  const dim3 grid = row_tile_grid(a.T, a.E, a.offsets, Tile::TM, ntiles);
  if (a.pre) hipLaunchKernelGGL((gemm_i8_dx_kernel<Tile, ODT, true>), grid, dim3(256 * Tile::GROUPS), 0, s, a, ntiles);
  else hipLaunchKernelGGL((gemm_i8_dx_kernel<Tile, ODT, false>), grid, dim3(256 * Tile::GROUPS), 0, s, a, ntiles);
  return hipGetLastError();
}
template <int ODT>
static int launch_dx(const GradI8Args& a, hipStream_t s) {
  const int side = tile_side(1, a.T, a.K);
  if (side == 256) return launch_dx_tile<TileGrad<false, 256, 256>, ODT>(a, s);
  if (side == 128) return launch_dx_tile<TileGrad<false, 128, 128>, ODT>(a, s);
  return launch_dx_tile<TileGrad<false, 64, 64>, ODT>(a, s);
}
int launch_gemm_i8_dx(const GradI8Args& a, hipStream_t s) {
  return a.out_dt == kBF16 ? launch_dx<kBF16>(a, s) : launch_dx<kF32>(a, s);
}

template <class Tile, int ODT>
static hipError_t launch_dw_tile(const GradI8Args& a, int splits, hipStream_t s) {
  const int kt = (a.K + Tile::TM - 1) / Tile::TM, nt = (a.N + Tile::TN - 1) / Tile::TN;
  const int most = (kt * nt * splits + kNumQueues - 1) / kNumQueues;
  const int64_t n = (int64_t)most * a.E * kNumQueues, x = std::min<int64_t>(n, 1 << 20);
  hipLaunchKernelGGL((gemm_i8_dw_kernel<Tile, ODT>), dim3((uint32_t)x, (uint32_t)((n + x - 1) / x)), dim3(256 * Tile::GROUPS), 0, s, a, kt, nt,
                     splits);
  return hipGetLastError();
}
template <int ODT>
static int launch_dw(const GradI8Args& a, hipStream_t s) {
  const int splits = dw_splits(a.E, a.T, a.N, a.K);
  if (splits > 1) {
    GradI8Args b = a;
    b.out = a.part;
    const hipError_t e = launch_dw_tile<TileGrad<true, 256, 256>, kF32>(b, splits, s);
    if (e != hipSuccess) return e;
    const int64_t n = (int64_t)a.E * a.K * a.N;
    hipLaunchKernelGGL(dw_sum_kernel<ODT>, dim3((uint32_t)std::min<int64_t>((n + 1023) / 1024, 8192)), dim3(256), 0, s, a.part,
                       a.out, n, splits);
    return hipGetLastError();
  }
  const int side = tile_side(a.E, a.K, a.N);
  if (side == 256) return launch_dw_tile<TileGrad<true, 256, 256>, ODT>(a, 1, s);
  if (side == 128) return launch_dw_tile<TileGrad<true, 128, 128>, ODT>(a, 1, s);
  return launch_dw_tile<TileGrad<true, 64, 64>, ODT>(a, 1, s);
}
int launch_gemm_i8_dw(const GradI8Args& a, hipStream_t s) {
  return a.out_dt == kBF16 ? launch_dw<kBF16>(a, s) : launch_dw<kF32>(a, s);
}

}  // namespace hocf
