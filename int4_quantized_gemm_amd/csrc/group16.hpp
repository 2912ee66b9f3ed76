// The 16-lane layout of a 256-group, shared by the row kernels that quantize,
// normalize or differentiate whole rows (rotate.hip, norm.hip): butterflies
// over the registers of a lane, a transpose through LDS between the two halves
// of the index bits, and the 16 inputs of a lane as loaded.
#pragma once

#include "device_common.hpp"

namespace tp {

// A 256-group is held by one 16-lane row of the wave: lane l loads elements
// 16 l + i (i = 0..15, index bits 0-3 in registers) and applies the four
// butterfly stages of those bits; the row then transposes the group through
// LDS so that lane l holds elements l + 16 r (bits 4-7 in registers) and
// applies the other four stages. Outputs stay in that order; the codes go back
// through LDS to be stored 16 contiguous bytes per lane.

// Four butterfly stages over the register index of 16 values.
template <typename T>
__device__ __forceinline__ void fwht16_regs(T (&v)[16]) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i & h) == 0) {
        const T a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
}

// Orders this wave's LDS writes before its later LDS reads (one wave: the LDS
// unit runs its operations in order; this keeps the compiler from reordering).
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_wave_barrier();
}

// Row transpose: lane l gives elements 16 l + i, receives elements l + 16 r.
// buf: this row's LDS area, touched by its 16 lanes only. Element e sits at
// e + PAD * (e / 16) so that neither side of the exchange has bank conflicts.
template <typename T>
__device__ __forceinline__ void transpose16(T (&v)[16], T* buf, int l16) {
  constexpr int PAD = sizeof(T) == 4 ? 4 : 2;
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < 16; ++i) buf[(16 + PAD) * l16 + i] = v[i];
  wave_lds_sync();
#pragma unroll
  for (int r = 0; r < 16; ++r) v[r] = buf[l16 + (16 + PAD) * r];
}

// The 16 inputs of one lane for one group, as loaded (bf16 pairs or fp32).
template <typename TIn>
struct Raw16;

template <>
struct Raw16<uint16_t> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float get(int i) const { return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
};

template <>
struct Raw16<float> {
  float w[16];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 f = reinterpret_cast<const float4*>(p)[c];
      w[4 * c] = f.x; w[4 * c + 1] = f.y; w[4 * c + 2] = f.z; w[4 * c + 3] = f.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0.f;
  }
  __device__ __forceinline__ float get(int i) const { return w[i]; }
};

// Largest magnitude of 16 doubles: a tree of v_max_f64 with both operands
// taken as magnitudes (one instruction per pair; written out because the
// compiler adds a canonicalizing max per element to fmax(., fabs(.))).
__device__ __forceinline__ double absmax2(double a, double b) {
  double r;
  asm("v_max_f64 %0, |%1|, |%2|" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

__device__ __forceinline__ double absmax16(const double (&v)[16]) {
  double m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = absmax2(v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
    for (int i = 0; i < w; ++i) m[i] = absmax2(m[i], m[i + w]);  // operands already >= 0
  return m[0];
}

}  // namespace tp
