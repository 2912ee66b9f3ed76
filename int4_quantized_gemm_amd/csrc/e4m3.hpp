// Codes of the 8-bit floating-point format e4m3 (OCP: 4 exponent bits with bias
// 7, 3 mantissa bits, subnormals, no infinity, largest value 448) for fp64
// quotients, rounded to nearest even and saturated.
#pragma once

#include "device_common.hpp"

namespace tp {

constexpr double E4M3_MAX = 448.0;

// The scale of a block: fp32(amax / 448), 0 for a block of zeros. For an fp32
// amax the fp64 product with 1 / 448 rounds to the same: amax / 448 = amax / 7 /
// 64 is no nearer than 2^-28 of itself to the middle of two fp32 numbers, unless
// it is an fp32 number.
__device__ __forceinline__ float e4m3_scale(double amax) { return (float)(amax / E4M3_MAX); }
__device__ __forceinline__ float e4m3_scale(float amax) { return (float)((double)amax * (1.0 / E4M3_MAX)); }

// The code of q. With e the exponent of |q| (at least -6, where the subnormal
// codes begin), |q| 2^(3 - e) is below 16 and its nearest integer n is the
// mantissa with its leading bit: the code is 8 (e + 6) + n, carries into the
// next exponent included.
__device__ __forceinline__ uint32_t e4m3_code(double q) {
  constexpr double MAGIC = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer (RNE)
  const uint64_t u = __builtin_bit_cast(uint64_t, q);
  const uint32_t hi = (uint32_t)(u >> 32) & 0x7fffffffu;
  const int e = max((int)(hi >> 20) - 1023, -6);
  const uint32_t scaled = hi + ((uint32_t)(3 - e) << 20);  // (zero and what is far below stay far below 1)
  const double r = __builtin_bit_cast(double, ((uint64_t)scaled << 32) | (uint32_t)u);
  const uint32_t n = (uint32_t)__builtin_bit_cast(uint64_t, r + MAGIC);
  const uint32_t code = min((uint32_t)(8 * (e + 6)) + n, 126u);
  return code | ((uint32_t)(u >> 56) & 0x80u);
}

// What the quick way of codes needs of a scale: 1 / s from below and from above.
// It takes x in fp32: from s = 2^-100 on, what fp32 holds as a subnormal is below
// 2^-26 s, so its code is 0 whatever its rounding; up to 2^118, 448 s and a bit is
// an fp32 number. Beyond, both are 0 and every code is decided by the division
// (slow).
struct E4m3Inverse {
  float s, lo, hi;
  __device__ __forceinline__ bool slow() const { return lo == 0.f && s > 0.f; }
};

__device__ __forceinline__ E4m3Inverse e4m3_inverse(float s) {
  const float inv = s >= 0x1p-100f && s <= 0x1p118f ? __builtin_amdgcn_rcpf(s) : 0.f;
  return E4m3Inverse{s, inv * (1.f - 0x1p-21f), inv * (1.f + 0x1p-21f)};
}

// The codes of N values, four to a dword: x(i) in fp32, exact(i) the value itself
// in fp64 (x(i) is it, or it rounded), of(i) its scale, slow whether any of those
// is. Rounding is monotone: the products with 1 / s from below and from above
// enclose x / s (the roundings of x, of the factor and of the product, 2^-24 each,
// and 1 / s, 2^-23, stay below 2^-21 together), so where both round to one code it
// is that of x / s. Where they do not the fp64 division decides: one value in 10^5 of
// fp32 data, one wave in 160; one in 200 of bf16 data, two waves in three (x / s is a
// midpoint itself where the 8 bits of the block's largest value are a multiple of 7).
// NaN, and infinity under its infinite scale, have a NaN code either way.
template <int N, typename X, typename D, typename S>
__device__ __forceinline__ void e4m3_codes(uint32_t (&w)[N / 4], X x, D exact, S of, bool slow) {
  uint32_t up[N / 4];
  bool open = slow;
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    int lo = 0, hi = 0;
    {
      const E4m3Inverse a = of(4 * q), b = of(4 * q + 1);
      const float u = x(4 * q), v = x(4 * q + 1);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(u * a.lo, v * b.lo, lo, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(u * a.hi, v * b.hi, hi, false);
    }
    {
      const E4m3Inverse a = of(4 * q + 2), b = of(4 * q + 3);
      const float u = x(4 * q + 2), v = x(4 * q + 3);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(u * a.lo, v * b.lo, lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(u * a.hi, v * b.hi, hi, true);
    }
    w[q] = (uint32_t)lo;
    up[q] = (uint32_t)hi;
    open |= lo != hi;
  }
  if (__ballot(open)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const E4m3Inverse a = of(i);
      const uint32_t mask = 0xffu << (8 * (i & 3));
      if (((w[i >> 2] ^ up[i >> 2]) & mask) != 0 || a.slow())
        w[i >> 2] = (w[i >> 2] & ~mask) | (e4m3_code(exact(i) / (double)a.s) << (8 * (i & 3)));
      __builtin_amdgcn_sched_barrier(0);  // one division at a time
    }
    if (__ballot(slow)) {  // (apart: in the division's way it took 3% more for every row)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (of(i).slow() && !(fabs(exact(i)) < __builtin_inf())) w[i >> 2] |= 0x7fu << (8 * (i & 3));
    }
  }
}

}  // namespace tp
