// Reductions over 16 or 64 lanes: pairs, quads, halves and rows of 16 by lane
// permutes inside the vector instructions, then by swaps of rows and halves.
#pragma once

#include "common.hpp"

namespace hocf {

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true);  // (folds into the instruction that uses it)
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, v)));
}
// The two values of a lane's pair of rows (SWAP = 16) or of halves (32), each
// the same in all 16 lanes of a row (or 32 of a half).
template <int SWAP>
__device__ __forceinline__ void across(uint32_t v, uint32_t& a, uint32_t& b) {
  const auto r = SWAP == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                            : __builtin_amdgcn_permlane32_swap(v, v, false, false);
  a = r[0];
  b = r[1];
}
template <class T, class OP>
__device__ __forceinline__ T across_rows(T v, OP op) {
  uint32_t a, b;
  across<16>(__builtin_bit_cast(uint32_t, v), a, b);
  v = op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
  across<32>(__builtin_bit_cast(uint32_t, v), a, b);
  return op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
}
template <int LPT>
__device__ __forceinline__ int row_max(int v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  v = max(v, dpp<0x140>(v));
  if constexpr (LPT == 64) v = across_rows(v, [](int a, int b) { return max(a, b); });
  return v;
}
template <int LPT>
__device__ __forceinline__ float row_maxf(float v) {
  v = fmaxf(v, dppf<0xB1>(v));
  v = fmaxf(v, dppf<0x4E>(v));
  v = fmaxf(v, dppf<0x141>(v));
  v = fmaxf(v, dppf<0x140>(v));
  if constexpr (LPT == 64) v = across_rows(v, [](float a, float b) { return fmaxf(a, b); });
  return v;
}
template <int LPT>
__device__ __forceinline__ float row_sum(float v) {
  v += dppf<0xB1>(v);
  v += dppf<0x4E>(v);
  v += dppf<0x141>(v);
  v += dppf<0x140>(v);
  if constexpr (LPT == 64) v = across_rows(v, [](float a, float b) { return a + b; });
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t row_add(uint32_t u) {
  int v = (int)u;
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  if constexpr (LPT == 64) v = across_rows(v, [](int a, int b) { return a + b; });
  return (uint32_t)v;
}

}  // namespace hocf
