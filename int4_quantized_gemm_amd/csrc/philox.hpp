// The mask of a dropout, computed where it is needed and never stored:
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
// as 1, 2, 3", 2011), a keyed bijection of a 128-bit counter. One call serves a
// run of eight elements of a row, 16 bits each:
//
//   key      the two halves of the seed
//   counter  the run's number in the matrix, row ceil(k / 8) + column / 8
//            (64 bits), then the offset (64 bits)
//   element  j of the run: bits 16 (j & 1) .. + 15 of word j / 2; it is kept
//            where they are at least the threshold round(65536 p)
//
// 16 bits an element and not 32: half the multiplications (Philox's ten rounds
// are 20 32 x 32 bit products), at a probability off by at most 2^-17, which the
// factor 65536 / (65536 - threshold) takes into account exactly.
#pragma once

#include "block_ops.hpp"
#include "device_common.hpp"

namespace tp {

struct PhiloxKey {
  uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ PhiloxKey philox_key(const uint64_t* rng) {
  const uint64_t s = rng[0], o = rng[1];
  return PhiloxKey{(uint32_t)s, (uint32_t)(s >> 32), (uint32_t)o, (uint32_t)(o >> 32)};
}

__device__ __forceinline__ u32x4_t philox4x32_10(const PhiloxKey& key, uint64_t run) {
  uint32_t a = (uint32_t)run, b = (uint32_t)(run >> 32), c = key.o0, d = key.o1;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
    a = (uint32_t)(q >> 32) ^ b ^ k0;
    b = (uint32_t)q;
    c = (uint32_t)(p >> 32) ^ d ^ k1;
    d = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{a, b, c, d};
}

// Whether element j (0 .. 7) of a run is kept.
__device__ __forceinline__ bool philox_keeps(const u32x4_t& w, int j, uint32_t threshold) {
  return ((w[j >> 1] >> (16 * (j & 1))) & 0xffffu) >= threshold;
}

// x scaled where it is kept, 0 where not (NaN and infinity too): the product
// rounded once, whatever is added to it.
__device__ __forceinline__ float philox_drop(const u32x4_t& w, int j, const DropArg& d, float x) {
#pragma clang fp contract(off)
  const float y = x * d.scale;
  return philox_keeps(w, j, d.threshold) ? y : 0.f;
}

}  // namespace tp
