// Codes of the 8-bit floating-point format e4m3 (OCP: 4 exponent bits with bias
// 7, 3 mantissa bits, subnormals, no infinity, largest value 448) for fp64
// quotients, rounded to nearest even and saturated.
#pragma once

#include "device_common.hpp"

namespace tp {

constexpr double E4M3_MAX = 448.0;

// The scale of a block: fp32(amax / 448), 0 for a block of zeros.
__device__ __forceinline__ float e4m3_scale(double amax) { return (float)(amax / E4M3_MAX); }

// The code of q. With e the exponent of |q| (at least -6, where the subnormal
// codes begin), |q| 2^(3 - e) is below 16 and its nearest integer n is the
// mantissa with its leading bit: the code is 8 (e + 6) + n, carries into the
// next exponent included. near is set where |q| is within 1e-9 of a tie of its
// binade's steps: there a quotient formed as x * (1 / s) may be on the other
// side of it than x / s.
__device__ __forceinline__ uint32_t e4m3_code(double q, bool& near) {
  constexpr double MAGIC = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer (RNE)
  const uint64_t u = __builtin_bit_cast(uint64_t, q);
  const uint32_t hi = (uint32_t)(u >> 32) & 0x7fffffffu;
  const int e = max((int)(hi >> 20) - 1023, -6);
  const uint32_t scaled = hi + ((uint32_t)(3 - e) << 20);  // (zero and what is far below stay far below 1)
  const double r = __builtin_bit_cast(double, ((uint64_t)scaled << 32) | (uint32_t)u);
  const double f = r + MAGIC;
  const double d = r - (f - MAGIC);
  near |= !(fabs(d) < 0.5 - 1e-9);
  const uint32_t n = (uint32_t)__builtin_bit_cast(uint64_t, f);
  const uint32_t code = min((uint32_t)(8 * (e + 6)) + n, 126u);
  return code | ((uint32_t)(u >> 56) & 0x80u);
}

// The codes of N values x(i) with their scales s(i) and inv(i) = 1 / s(i) (0
// where s(i) is 0), four to a dword. The ones that lie next to a tie are decided
// by the division itself (one wave in a hundred takes it on random values).
template <int N, typename X, typename S, typename I>
__device__ __forceinline__ void e4m3_codes(uint32_t (&w)[N / 4], X x, S s, I inv) {
  bool near = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t c = e4m3_code(x(i) * inv(i), near);
    w[i >> 2] = (i & 3) == 0 ? c : w[i >> 2] | (c << (8 * (i & 3)));
  }
  if (__ballot(near)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      bool tie = false, again = false;
      e4m3_code(x(i) * inv(i), tie);
      if (tie && inv(i) > 0.0) {
        const uint32_t c = e4m3_code(x(i) / (double)s(i), again);
        w[i >> 2] = (w[i >> 2] & ~(0xffu << (8 * (i & 3)))) | (c << (8 * (i & 3)));
      }
      __builtin_amdgcn_sched_barrier(0);  // one division at a time
    }
  }
}

}  // namespace tp
