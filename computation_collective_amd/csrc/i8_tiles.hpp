// What the 8-bit products and their gradients share: the tiles of grouped rows,
// LDS layouts of tile stages, and loads straight into them.
#pragma once

#include <algorithm>

#include "i8.hpp"
#include "lanes.hpp"
#include "mfma_tile.hpp"
#include "publish.hpp"
#include "sync.hpp"

namespace hocf {

#if defined(__HIP_DEVICE_COMPILE__)
#define HOCF_LDS __attribute__((address_space(3)))
#else
#define HOCF_LDS
#endif

// A buffer resource over [base, base + bytes): loads past its end give zeros and
// touch no memory (base and bytes wave-uniform, bytes < 2^31).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t ranged_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, kRawBufferWord3);
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past the end of every resource

// 16 bytes a lane from voff (per lane) + soff (wave-uniform) to 1 KB of LDS.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (HOCF_LDS void*)lds, 16, (int)voff, uniform((int)soff), 0, 0);
#endif
}

// The memory operations before it are issued before those after it: a count of
// operations still on their way says which they are.
__device__ __forceinline__ void in_order() { __asm__ volatile("" ::: "memory"); }

// vmcnt(N) and lgkmcnt(0), then the workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  static_assert(N <= 63, "vmcnt range");
  in_order();
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
  in_order();
  __builtin_amdgcn_s_barrier();
  in_order();
}

// Order within a quarter of a step: NM matrix instructions, ND LDS reads soon behind the
// first of them, NL loads, NV vector instructions and NW LDS writes spread over all.  Nothing moves
// out of the quarter: counts of loads on their way go by it.
template <int NM, int ND, int NL, int NV, int NW, int X = 0>
__device__ __forceinline__ void mix() {
  if constexpr (X < NM) {
    constexpr int dpm = (ND + NM - 1) / NM, d = ND - X * dpm < dpm ? (ND - X * dpm > 0 ? ND - X * dpm : 0) : dpm;
    constexpr int l = NL * (X + 1) / NM - NL * X / NM, v = NV * (X + 1) / NM - NV * X / NM, w = NW * (X + 1) / NM - NW * X / NM;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
    if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(0x020, l, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x002, v, 0);
    if constexpr (w > 0) __builtin_amdgcn_sched_group_barrier(0x200, w, 0);
    mix<NM, ND, NL, NV, NW, X + 1>();
  } else {
    in_order();
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Steps 0 .. n - 1 and on to whole turns of a ring of four stages, each step with its stage as a
// constant.  (No way out in between: it would cost copies of the accumulators and of what is being loaded.)
template <class S>
__device__ __forceinline__ void four_steps(int n, S step) {
  for (int ks = 0; ks < n; ks += 4) {
    step(std::integral_constant<int, 0>{}, ks);
    step(std::integral_constant<int, 1>{}, ks + 1);
    step(std::integral_constant<int, 2>{}, ks + 2);
    step(std::integral_constant<int, 3>{}, ks + 3);
  }
}

// An offset within [0, T] (T < 2^31).
__device__ __forceinline__ int within(int64_t o, int64_t T) { return (int)(o < 0 ? 0 : o > T ? T : o); }

// Group bounds, whatever the offsets hold: each counts as the largest of itself and those before it, within
// [0, T].  So groups follow one another and share no row, also where the offsets fall.

// Of one group e (uniform).  Every lane takes part.
__device__ __forceinline__ void group_bounds(const int64_t* offsets, int e, int64_t T, int64_t* lo, int64_t* hi) {
  int m = 0;
  for (int i = threadIdx.x & 63; i - (int)(threadIdx.x & 63) <= e; i += 256) {
#pragma unroll
    for (int u = 0; u < 256; u += 64) m = max(m, within(offsets[min(i + u, e)], T));
  }
  m = uniform(row_max<64>(m));
  *lo = m;
  *hi = max(m, within(offsets[e + 1], T));
}

// Of groups e0 + lane, 64 at a time (past the last: no rows).  Only where some offset of the list falls or leaves
// [0, T] (`fall`, uniform) do those before e0 matter: `upto` is their largest, 0 at first.  Whether this
// group's own do.
__device__ __forceinline__ bool lane_bounds(const int64_t* offsets, int E, int64_t T, int e0, bool fall, int* upto, int* lo,
                                            int* hi) {
  const int lane = threadIdx.x & 63, e = min(e0 + lane, E);
  const int64_t a = offsets[e], b = offsets[min(e + 1, E)];
  *lo = within(a, T);
  *hi = max(*lo, within(b, T));
  const bool own = *lo != a || *hi != b;
  if (fall) {
    int m = max(*hi, *upto);
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(m, d, 64);
      if (lane >= d) m = max(m, o);
    }
    const int before = __shfl_up(m, 1, 64);
    *lo = lane ? before : max(*lo, *upto);
    *hi = m;
    *upto = uniform(__shfl(m, 63, 64));
  }
  return own;
}

struct RowTile {
  int64_t row, end;  // first row, and the end of its group
  int e, nt;         // expert and column tile; e = -1: none
};

// Workgroup b's tile of TM rows x one of `ntiles` columns.  The groups' row tiles stand one
// after another; each XCD (workgroups are dealt to them in turn) takes one run of all tiles, in blocks of
// up to 8 column tiles, row tile by row tile, so that what it reads together shares its L2.
// Every wave finds the same.  Offsets that fall or leave [0, T] are reported by workgroup 0.
template <int TM>
__device__ __forceinline__ RowTile row_tile(const int64_t* offsets, int E, int64_t T, int ntiles, const SyncArgs& sync) {
  const int lane = threadIdx.x & 63;
  RowTile t{0, T, 0, 0};
  int64_t total, skip = 0;
  bool fall = false;
  auto tiles = [](int lo, int hi) { return (int)(((uint32_t)(hi - lo) + TM - 1) / TM); };
  if (!offsets) {
    total = (T + TM - 1) / TM;
  } else {
    int n = 0, upto = 0, lo, hi;
    bool own = false;
    for (int e0 = 0; e0 < E; e0 += 64) {
      own |= lane_bounds(offsets, E, T, e0, false, &upto, &lo, &hi);
      n += tiles(lo, hi);
    }
    fall = __ballot(own) != 0;
    if (fall) {
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report_status(sync, kErrBadIndex);
      n = 0;
      for (int e0 = 0; e0 < E; e0 += 64) {
        lane_bounds(offsets, E, T, e0, true, &upto, &lo, &hi);
        n += tiles(lo, hi);
      }
    }
    for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d, 64);
    total = n;
  }
  total = uniform64(total) * ntiles;
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;  // (a row of the grid is whole turns of the XCDs)
  const int q = (int)(b % kNumQueues);
  const int64_t at = total * q / kNumQueues + b / kNumQueues;
  if (at >= total * (q + 1) / kNumQueues) {
    t.e = -1;
    return t;
  }
  int64_t mtiles = total / ntiles;
  if (offsets) {
    // the group that holds tile `at`: tiles before it are skip * ntiles
    bool found = false;
    int last = 0;
    for (int e0 = 0; e0 < E && !found; e0 += 64) {
      int lo, hi;
      lane_bounds(offsets, E, T, e0, fall, &last, &lo, &hi);
      const int n = tiles(lo, hi);
      int upto = n;
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d, 64);
        if (lane >= d) upto += o;
      }
      const uint64_t m = __ballot((skip + upto) * (int64_t)ntiles > at);
      if (m) {
        const int l = __builtin_ctzll(m);
        t.e = uniform(e0 + l);
        skip = uniform64(skip + __shfl(upto, l, 64) - __shfl(n, l, 64));
        mtiles = uniform(__shfl(n, l, 64));
        t.row = uniform(__shfl(lo, l, 64));
        t.end = uniform(__shfl(hi, l, 64));
        found = true;
      } else {
        skip = uniform64(skip + __shfl(upto, 63, 64));
      }
    }
  }
  const int64_t j = at - skip * ntiles;
  constexpr int kColBlock = 8;
  const int64_t block = mtiles * kColBlock;
  const int nb = (int)(j / block), width = min(kColBlock, ntiles - nb * kColBlock);
  const int64_t in = j - nb * block;
  t.row += in / width * TM;
  t.nt = nb * kColBlock + (int)(in % width);
  t.e = uniform(t.e);
  t.nt = uniform(t.nt);
  t.row = uniform64(t.row);
  return t;
}

// The side of the tiles for `groups` results of rows x columns each: 256 where its tiles fill five
// eighths of the turns of 256 CUs that they take, else 128 where there are enough of them, else 64.
// Measured with 256 and 128 (in brackets the tiles of 256): 8-bit product 4096 x 1024 -> 2048
// (128) 21.8 and 14.3 us, 6144 x 4096 -> 1792 (168) 58.6 and 60.6, 9216 x 2048 -> 2048 (288) 63 and 52,
// 8192 x 8192 -> 8192 (1024) 439 and 496; dx 4096 x 1024 -> 2048 34 and 26, 6144 x 4096 -> 1792 117
// and 131.  With 128 and 64 (the tiles of 128): product 2000 x 1024 -> 1024 (128) 7.4 and 6.5, 3000 x
// 2048 -> 1024 (192) 11.2 and 13.0; dx 1500 x 1000 -> 1040 (108) 14.7 and 13.1, 3000 x 2048 -> 1024
// (192) 26.8 and 34; dw 512 x 1536 x 1536 (144) 11.2 and 13.5.
// The products and dx count all rows as one group: with many short groups most of a tile may be padding.  Not
// measured against smaller sides; 8192 rows x 1024 -> 512 on 256 experts take 33 us (the weights' bytes 28),
// dx 55, and 16384 rows x 1024 -> 1792 on 64 experts 49 and 62.
inline int tile_side(int64_t groups, int64_t rows, int64_t columns) {
  const int64_t big = groups * ((rows + 255) / 256) * ((columns + 255) / 256);
  if (big * 8 >= (big + 255) / 256 * 256 * 5) return 256;
  return groups * ((rows + 127) / 128) * ((columns + 127) / 128) > 128 ? 128 : 64;
}

// Workgroups that cover the tiles of any offsets.
inline dim3 row_tile_grid(int64_t T, int E, bool grouped, int TM, int ntiles) {
  int64_t rows = (T + TM - 1) / TM;
  if (grouped) rows = std::min(T, T / TM + E);  // (a group ends at most one tile that is not full)
  const int64_t total = rows * ntiles;
  const int64_t n = (total + kNumQueues - 1) / kNumQueues * kNumQueues, x = std::min<int64_t>(n, 1 << 20);
  return dim3((uint32_t)x, (uint32_t)((n + x - 1) / x));
}

// A tile's results to memory, row by row: value(i, j, g) gives the four results of group g of
// block (i, j) (row 32 i + lane mod 32, columns 32 j + 8 g + 4 (lane / 32) .. of the wave's
// part) and finish(row, column, v) what becomes of four results of one row before they are
// rounded.  A wave stages 32 rows in LDS (FIN: in fp32, else as they are stored) and stores
// whole lines.  Rows < rows and columns < cols only (cols a multiple of 8).
template <class Tile, int ODT, bool FIN, class V, class F>
__device__ __forceinline__ void store_rows(char* dst, int64_t ld, int rows, int cols, char* const (&stages)[4], V value,
                                           F finish) {
  constexpr int SDT = FIN ? kF32 : ODT;
  using L = PublishLayout<Tile, SDT>;
  constexpr int OES = ODT == kBF16 ? 2 : 4, CE = 16 / L::ES;  // elements of a staged piece
  constexpr int RPI = 64 / L::NCH, NIT = L::NCH / 2;
  constexpr int BATCH = NIT < 8 ? NIT : 8;
  const int wave = uniform(threadIdx.x >> 6), lane = opaque_lane();
  const int wm = wave / Tile::WN, wn = wave % Tile::WN;
  const int lr = lane & 31, half = lane >> 5, sr = lane / L::NCH, sc = lane % L::NCH;
  const int tcol = wn * Tile::WTN + sc * CE;
  wait_barrier<0>();  // (loads past the sum's end may still be on their way into the stages)
  char* area = L::area(stages, wave);
#pragma unroll
  for (int i = 0; i < Tile::FM; ++i) {
#pragma unroll
    for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int byte = (32 * j + 8 * g + 4 * half) * L::ES;
        char* p = area + L::at(lr, byte >> 4) + (byte & 15);
        const floatx4 v = value(i, j, g);
        if constexpr (SDT == kBF16) *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else *reinterpret_cast<floatx4*>(p) = v;
      }
    // (LDS operations of one wave complete in order; the compiler must not reuse an earlier block's)
    __asm__ volatile("" ::: "memory");
#pragma unroll
    for (int it0 = 0; it0 < NIT; it0 += BATCH) {
      u32x4 v[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) v[b] = *reinterpret_cast<const u32x4*>(area + L::at((it0 + b) * RPI + sr, sc));
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int trow = wm * Tile::WTM + 32 * i + (it0 + b) * RPI + sr;
        if (trow < rows && tcol < cols) {
          char* p = dst + ((int64_t)trow * ld + tcol) * OES;
          if constexpr (FIN) st4<ODT>(p, 0, finish(trow, tcol, __builtin_bit_cast(floatx4, v[b])));
          else *reinterpret_cast<u32x4*>(p) = v[b];
        }
      }
    }
    __asm__ volatile("" ::: "memory");
  }
}

}  // namespace hocf
