// Launch-side declarations of the 8-bit integer operators (i8_abi.cpp checks
// the arguments, the i8_*.hip units launch).
#pragma once

#include <algorithm>

#include "internal.hpp"

namespace hocf {

enum Act : int { kNone = 0, kSilu = 1 };

constexpr int kI8MaxDim = 1 << 16;      // columns of a row of codes: 2^16 products of 2^14 stay below 2^31
constexpr int kI8MaxExperts = 1024;
constexpr int kI8MaxRows = 1024;        // rows of a decode product

// The smallest scale: a row's codes are its numbers over max(largest / 127, this).
constexpr float kI8TinyScale = 0x1p-126f;

struct QuantI8Args {
  const void* x;      // [T][ld] dt
  int8_t* codes;      // [T][K]
  float* scales;      // [T]
  int8_t* pre_codes;  // [T][K] or NULL: of x itself where codes are of act(x)
  float* pre_scales;  // [T] or NULL
  int64_t T, ld;
  int K, dt, act;
};

struct DequantI8Args {
  const int8_t* codes;  // [T][K]
  const float* scales;  // [T]
  void* out;            // [T][K] dt
  int64_t T;
  int K, dt;
};

struct WeightsI8Args {
  const void* W;       // [E][K][N] dt
  int8_t* wq;          // [E][N][K]
  float* scales;       // [E][N]
  uint32_t* part;      // workspace: [E][slabs][N] magnitudes (their bits)
  int E, N, K, dt, slabs;
};
constexpr int kW8SlabRows = 256;  // rows of W whose largest magnitudes one workgroup takes
inline int w8_slabs(int K) { return (K + kW8SlabRows - 1) / kW8SlabRows; }

struct GemmI8Args {
  const int8_t* xq;        // [T][K]
  const float* xs;         // [T]
  const int8_t* wq;        // [E][N][K]
  const float* ws;         // [E][N]
  const int64_t* offsets;  // [E + 1] or NULL (E = 1: every row)
  void* out;               // [T][N] out_dt
  int64_t T;
  int E, N, K, out_dt;
  SyncArgs sync;
};

struct GemvI8Args {
  const int8_t* xq;        // [R / rows_per_x][K]
  const float* xs;         // [R / rows_per_x]
  const int32_t* experts;  // [R] or NULL
  const int8_t* wq;        // [E][N][K]
  const float* ws;         // [E][N]
  void* out;               // [R][N] out_dt
  int R, rows_per_x, E, e0, N, K, out_dt;
};

struct GradI8Args {
  const uint16_t* dy;      // [T][N] bf16
  const int8_t* q;         // dx: the weights' codes [E][N][K]; dw: the rows' codes [T][K]
  const float* s;          // dx: [E][N]; dw: [T]
  const int64_t* offsets;  // [E + 1] or NULL (E = 1: every row)
  const int8_t* pre;       // dx: [T][K] or NULL
  const float* pre_s;      // dx: [T] or NULL
  void* out;               // dx: [T][K]; dw: [E][K][N], out_dt
  float* part;             // dw: workspace, [splits][E][K][N] where there are more than one
  int64_t T;
  int E, N, K, out_dt;
  SyncArgs sync;
};

// Parts that dw's sums over rows are taken in: as many as give each of 256 CUs a 256 x 256
// tile, where the tiles alone would leave half of them idle and each part is long enough to be worth its
// sums' way through memory.
inline int dw_splits(int E, int64_t T, int N, int K) {
  const int64_t tiles = (int64_t)E * ((K + 255) / 256) * ((N + 255) / 256);
  return (int)std::max<int64_t>(1, std::min<int64_t>(256 / tiles, T / E / 1024));
}

int launch_quant_i8(const QuantI8Args& a, hipStream_t s);
int launch_dequant_i8(const DequantI8Args& a, hipStream_t s);
int launch_weights_i8(const WeightsI8Args& a, hipStream_t s);
int launch_gemm_i8(const GemmI8Args& a, hipStream_t s);
int launch_gemv_i8(const GemvI8Args& a, hipStream_t s);
int launch_gemm_i8_dx(const GradI8Args& a, hipStream_t s);
int launch_gemm_i8_dw(const GradI8Args& a, hipStream_t s);

}  // namespace hocf
