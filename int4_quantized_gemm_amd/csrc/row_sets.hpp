// The row layout of the norms (norm.hip, layernorm.hip): a 256-group is held by
// a set of 16 lanes, 16 elements each (two runs of eight, 128 apart), a row by
// one set per group, a block by one wide row or several short ones.
#pragma once

#include <type_traits>

#include "block_ops.hpp"
#include "group16.hpp"

namespace tp {

// Sum over the 16 lanes of a set: the same value in each of them (addition
// commutes, so the exchange gives every lane the same tree).
template <typename T>
__device__ __forceinline__ T set_sum(T v) {
  v += swz_xor<1>(v);
  v += swz_xor<2>(v);
  v += swz_xor<4>(v);
  v += swz_xor<8>(v);
  return v;
}

__device__ __forceinline__ double set_max(double v) {
  v = fmax(v, swz_xor<1>(v));
  v = fmax(v, swz_xor<2>(v));
  v = fmax(v, swz_xor<4>(v));
  v = fmax(v, swz_xor<8>(v));
  return v;
}

// The other half of transpose16 (lane l's element r becomes lane r's element
// l, and back).
template <typename T>
__device__ __forceinline__ void transpose16_back(T (&v)[16], T* buf, int l16) {
  constexpr int PAD = sizeof(T) == 4 ? 4 : 2;
  wave_lds_sync();
#pragma unroll
  for (int r = 0; r < 16; ++r) buf[l16 + (16 + PAD) * r] = v[r];
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = buf[(16 + PAD) * l16 + i];
}

// The 16 elements of a lane: two runs of eight, 128 apart, so that a set's
// loads and stores cover whole lines (one run of 16 took fp32 rows four partial
// stores a line: 20.7 against 15.8 us for the gradients of 333 x 12288).
template <typename T>
struct Runs;

template <>
struct Runs<uint16_t> {
  u32x4_t w[2];
  __device__ __forceinline__ void load(const uint16_t* p) {
    w[0] = *reinterpret_cast<const u32x4_t*>(p);
    w[1] = *reinterpret_cast<const u32x4_t*>(p + 128);
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = u32x4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t v = w[i >> 3][(i >> 1) & 3];
    return (i & 1) ? bf16_hi(v) : bf16_lo(v);
  }
};

template <>
struct Runs<float> {
  f32x4_t w[4];
  __device__ __forceinline__ void load(const float* p) {
    w[0] = *reinterpret_cast<const f32x4_t*>(p);
    w[1] = *reinterpret_cast<const f32x4_t*>(p + 4);
    w[2] = *reinterpret_cast<const f32x4_t*>(p + 128);
    w[3] = *reinterpret_cast<const f32x4_t*>(p + 132);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ float get(int i) const { return w[i >> 2][i & 3]; }
};

__device__ __forceinline__ void load_vec16(const VecArg& g, int64_t c, float (&v)[16]) {
  if (g.p == nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 1.0f;
  } else if (g.bf16) {
    Runs<uint16_t> r;
    r.load((const uint16_t*)g.p + c);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = r.get(i);
  } else {
    Runs<float> r;
    r.load((const float*)g.p + c);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = r.get(i);
  }
}

__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<f32x4_t*>(p + 128 * (c >> 1) + 4 * (c & 1)) =
        f32x4_t{v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]};
}

__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<u32x4_t*>(p + 128 * h) =
        u32x4_t{pack_bf16x2(v[8 * h], v[8 * h + 1]), pack_bf16x2(v[8 * h + 2], v[8 * h + 3]),
                pack_bf16x2(v[8 * h + 4], v[8 * h + 5]), pack_bf16x2(v[8 * h + 6], v[8 * h + 7])};
}

// A value as the stream type holds it.
template <typename TS>
__device__ __forceinline__ float as_stream(float v) {
  if constexpr (std::is_same<TS, float>::value)
    return v;
  else
    return bf16_lo(pack_bf16x2(v, 0.f));
}

// Where a thread sits: its set, the row of the block that the set works on and
// the group of that row. Rows of four groups and more take a block each, and
// their sets' partial results are joined by wave first; shorter rows share a
// block and are joined set by set.
struct Place {
  int l16, set, slot, grp, rows;  // rows: rows of a block
  bool wide, active;
};

__device__ __forceinline__ Place place_of(int groups, int rows_per_block) {
  Place p;
  p.l16 = threadIdx.x & 15;
  p.set = threadIdx.x >> 4;
  p.slot = p.set / groups;
  p.grp = p.set - p.slot * groups;
  p.rows = rows_per_block;
  p.wide = groups >= 4 && rows_per_block == 1;
  p.active = p.slot < rows_per_block;
  return p;
}

// How rows are dealt to blocks.
struct Shape {
  int rows;     // rows of a block
  int threads;  // whole waves
  int64_t blocks;
};

// Rows of fewer than four groups share a block of 16 sets; the others take a
// block each. max_blocks: blocks walk rows beyond that many.
inline Shape shape_of(int64_t m, int groups, int64_t max_blocks) {
  Shape s;
  s.rows = groups < 4 ? 16 / groups : 1;
  s.threads = (s.rows * groups * 16 + 63) / 64 * 64;
  s.blocks = (m + s.rows - 1) / s.rows;
  if (s.blocks > max_blocks) s.blocks = max_blocks;
  return s;
}

}  // namespace tp
