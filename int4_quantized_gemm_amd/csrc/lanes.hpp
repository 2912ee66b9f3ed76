// Sums and maxima across lanes on the vector unit (no trip through the LDS unit,
// as ds_swizzle takes): rotations within rows of 16 lanes, then swaps of rows.
// Every lane gets the same bits: each step adds the same two values everywhere
// they meet, and addition commutes.
#pragma once

#include "device_common.hpp"

namespace tp {

// The value of the lane N further on in the row of 16.
template <int N>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, true);
}
template <int N>
__device__ __forceinline__ float row_rotate(float v) {
  return __builtin_bit_cast(float, row_rotate<N>(__builtin_bit_cast(uint32_t, v)));
}
template <int N>
__device__ __forceinline__ double row_rotate(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = row_rotate<N>((uint32_t)u), hi = row_rotate<N>((uint32_t)(u >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The two values that meet where rows of 16 (ROW 16) or halves of the wave (32)
// are paired: a has the lower one's, b the upper one's, in the lanes of both.
template <int ROW>
__device__ __forceinline__ void paired(uint32_t v, uint32_t& a, uint32_t& b) {
  if constexpr (ROW == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  }
}
template <int ROW>
__device__ __forceinline__ void paired(float v, float& a, float& b) {
  uint32_t x, y;
  paired<ROW>(__builtin_bit_cast(uint32_t, v), x, y);
  a = __builtin_bit_cast(float, x);
  b = __builtin_bit_cast(float, y);
}
template <int ROW>
__device__ __forceinline__ void paired(double v, double& a, double& b) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  uint32_t al, bl, ah, bh;
  paired<ROW>((uint32_t)u, al, bl);
  paired<ROW>((uint32_t)(u >> 32), ah, bh);
  a = __builtin_bit_cast(double, ((uint64_t)ah << 32) | al);
  b = __builtin_bit_cast(double, ((uint64_t)bh << 32) | bl);
}

template <bool MAX, typename T>
__device__ __forceinline__ T meet(T a, T b) {
  if constexpr (!MAX)
    return a + b;
  else if constexpr (sizeof(T) == 8)
    return fmax(a, b);
  else
    return fmaxf(a, b);
}

// Over rows of 16 lanes.
template <bool MAX, typename T>
__device__ __forceinline__ T row_all(T v) {
  v = meet<MAX>(v, row_rotate<8>(v));
  v = meet<MAX>(v, row_rotate<4>(v));
  v = meet<MAX>(v, row_rotate<2>(v));
  return meet<MAX>(v, row_rotate<1>(v));
}

// Over the four lanes of all rows that have the same place in them.
template <bool MAX, typename T>
__device__ __forceinline__ T rows_all(T v) {
  T a, b;
  paired<16>(v, a, b);
  v = meet<MAX>(a, b);
  paired<32>(v, a, b);
  return meet<MAX>(a, b);
}

}  // namespace tp
