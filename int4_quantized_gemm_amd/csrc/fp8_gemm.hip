// Product of two e4m3 matrices with a scale for each block of 128 along k:
//
//   C[i, c] = sum_g sa[g, i] sb(g, c) sum_{q in block g} a[i, q] b[c, q]
//
// sb one number per 128 x 128 block of b (weights), or per row of b and block
// (an operand that was quantized like a, as in a weight's gradient).
//
// A block of k starts from zero on the matrix unit, and its fp32 result is folded
// into the fp32 sums with the product of the two scales, on the vector unit
// beside the next instructions. Two ways to sum a block:
//   bf16 C   one 16x16x128 8-bit float instruction. It adds eight products at a
//            time aligned to the largest of them and drops what lies below about
//            2^-15 of it (measured: 1.3e-5 of the result's norm on Gaussian
//            codes, 3.3e-5 with one channel 100 times the others, 3.6e-5 with one
//            in 200 30 times, where 2.2% of the results round the other way): far
//            inside bf16's own rounding, 1.7e-3 of the norm, not inside fp32's.
//   fp32 C   four 16x16x32 bf16 instructions on the widened codes (exact), whose
//            sums are fp32's; half the matrix rate.
// The instruction's first operand is b and its second a, so that a lane holds
// consecutive columns of one row of C and needs one scale of a per fragment.
// Fragment j of a wave takes the rows 4 FN (r / 4) + 4 j + r % 4 of its share
// of b, r = 0 .. 15, which makes the columns a lane holds 4 FN consecutive ones.
//
// LDS: rows of 128 bytes, 16-byte granules; granule c of a row sits at c ^ f,
// f from two bits of the row chosen so that the 16 lanes that ds_read_b128
// serves together touch 16 different granules of 256 bytes (gemm_pp.hpp).
#include <algorithm>

#include "block_ops.hpp"
#include "gemm_pp.hpp"

namespace tp {

typedef __attribute__((ext_vector_type(8))) int i32x8_t;

namespace {

// 16 x 16 results over 128 of k, from zero.
__device__ __forceinline__ f32x4_t mfma_e4m3(i32x8_t first, i32x8_t second) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(first, second, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// Eight codes (two dwords) as bf16, exact.
__device__ __forceinline__ bf16x8_t widen_e4m3(int lo, int hi) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// The 32 codes of a lane, as the matrix instructions take them.
template <bool EXACT>
struct Frag;

template <>
struct Frag<false> {
  i32x8_t v;
  __device__ __forceinline__ void set(i32x8_t codes) { v = codes; }
};

template <>
struct Frag<true> {
  bf16x8_t v[4];
  __device__ __forceinline__ void set(i32x8_t codes) {
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = widen_e4m3(codes[2 * s], codes[2 * s + 1]);
  }
};

// One fragment of a against FN of b, over a block, from zero.
template <int FN>
__device__ __forceinline__ void block_sums(const Frag<false> (&b)[FN], const Frag<false>& a, f32x4_t (&p)[FN]) {
#pragma unroll
  for (int j = 0; j < FN; ++j) p[j] = mfma_e4m3(b[j].v, a.v);
}

template <int FN>
__device__ __forceinline__ void block_sums(const Frag<true> (&b)[FN], const Frag<true>& a, f32x4_t (&p)[FN]) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      p[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j].v[s], a.v[s], s ? p[j] : f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
}

__device__ __forceinline__ i32x8_t join8(u32x4_t lo, u32x4_t hi) {
  return i32x8_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// The exponent of a scale and its side's bias: at most MID_SCALES for a scale of a
// within 2^-85 .. 2^40, one of b within 2^-41 .. 2^84, or 0 (infinity and NaN too, whose
// products show whatever way they take). The product of two such is 0 because one of
// them is, or a normal number. (a has the room below: in the gradients it is the
// smaller side. The least and the largest of either side, looked at together, leave
// more room and took 2 to 5% more, in every product.)
constexpr uint32_t MID_SCALES = 124;
constexpr int A_BIAS = 84, B_BIAS = 40;
__device__ __forceinline__ uint32_t scale_reach(float s, int bias) {
  return (uint32_t)(__builtin_amdgcn_frexp_expf(s) + bias);  // s is 0.5 .. 1 times 2^it
}

// A block's sum folded into the results where its scales may not be such: a block's
// sum is 0 or within 2^-18 .. 2^25, so p sa sb is often an ordinary number where fp32
// holds sa sb as a subnormal, as 0 or as infinity. There fp64 holds all of it. Where
// the product is a normal number the bits are those of the usual way: a row's
// results do not depend on its neighbours' scales.
__device__ __forceinline__ float fold_wide(float p, float sa, float sb, float c) {
  const float s = sa * sb;
  if (__builtin_isnormal(s)) return fmaf(p, s, c);
  return (float)fma((double)p * (double)sa, (double)sb, (double)c);
}

// N consecutive columns of a row of C, as far as it has them.
template <int N, typename T>
__device__ __forceinline__ void store_cols(T* p, int left, bool vec, const float (&v)[N]) {
  if (vec && left >= N) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < N; e += 4) *reinterpret_cast<f32x4_t*>(p + e) = f32x4_t{v[e], v[e + 1], v[e + 2], v[e + 3]};
    } else if constexpr (N % 8 == 0) {
#pragma unroll
      for (int e = 0; e < N; e += 8)
        *reinterpret_cast<u32x4_t*>(p + e) = u32x4_t{pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]),
                                                     pack_bf16x2(v[e + 4], v[e + 5]), pack_bf16x2(v[e + 6], v[e + 7])};
    } else {
#pragma unroll
      for (int e = 0; e < N; e += 4)
        *reinterpret_cast<uint2*>(p + e) = uint2{pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < left) {
        if constexpr (sizeof(T) == 4)
          p[e] = v[e];
        else
          p[e] = (uint16_t)pack_bf16x2(v[e], 0.f);
      }
  }
}

}  // namespace

// Schedule. Two stages of one block of k (128 bytes a row, and the scales) in LDS:
// direct loads fill one while the other is worked on, one barrier a step. The
// scales come the same way: a load to registers would have to be waited for, and
// with it, in order, every direct load before it (256 x 256 tiles, 4096 x 12288
// x 4096: 258 us with the scale of b loaded so, 200 through LDS). A wave reads
// its fragments of b once a step and each of a one ahead of its use, and issues a
// matrix instruction with the vector work of the previous fragment in its shadow.
// Measured, calls in a row: 4096 x 12288 x 4096, bf16 C, 198 us, 2080 TFLOP/s (the
// instruction alone 3800; 214 us between other kernels); 2000 x 4096 x 4096 39.5 us,
// 1700. With an fp32 C 4096 x 4096 x 4096 140 us, 980, and with a scale a row of b
// and k 2048 89 us, 770 (the bf16 instruction alone 1830): there the widening and the
// folds, 3.5 to 4.5 vector instructions beside each matrix instruction, are the bound
// (two of them are free, four make a bf16 instruction 11.8 ns instead of 7.9, two
// waves a SIMD; beside an 8-bit one of 14.3 ns four make 16.3); widening each fragment
// of a beside the products of the one before changed nothing (88 us).
template <int BM, int BN, int WM, int WN, int NS>
struct F8Cfg {
  static constexpr int NWN = BN / WN, NW = (BM / WM) * NWN, NT = 64 * NW;
  static constexpr int FM = WM / 16, FN = WN / 16;
  static constexpr int A_BYTES = BM * 128, AB_BYTES = (BM + BN) * 128;
  static constexpr int STAGE = AB_BYTES + 4 * (BM + BN);  // operands, then their scales
  static constexpr int LOADS = (BM + BN) / 8, LPW = LOADS / NW;  // direct loads of 1 KB
  static constexpr int LDS_BYTES = NS * STAGE;
  static_assert(LOADS % NW == 0 && BM % 64 == 0 && BN % 64 == 0 && 128 % WN == 0, "whole loads, one block of b a wave");
  static_assert((BM + BN) / 64 <= NW && LDS_BYTES <= 160 * 1024, "a load of scales a wave");
  static_assert((NS & (NS - 1)) == 0 && (NS - 2) * (LPW + 1) < 64, "ring and vmcnt");
  static_assert(BN % 128 == 0, "tiles begin with a block of b");
};

// PARTIAL: the steps [blockIdx.y * sps, ..) of k, raw sums to part.
template <int BM, int BN, int WM, int WN, int NS, bool BROWS, bool OUT_BF16, bool PARTIAL>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), 2) void k_qgemm_fp8(GemmFp8Args g, int tiles_m, int tiles_n,
                                                                            int gm, int sps, int64_t ldp) {
  using Cfg = F8Cfg<BM, BN, WM, WN, NS>;
  constexpr int FM = Cfg::FM, FN = Cfg::FN, LPW = Cfg::LPW;
  extern __shared__ __align__(1024) uint8_t ring[];
  int tm, tn;
  pp_map_tile(blockIdx.x, gridDim.x, tiles_m, tiles_n, gm, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int M = (int)g.m, N = (int)g.n;
  const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm0 = (wave / Cfg::NWN) * WM, wn0 = (wave % Cfg::NWN) * WN;
  auto swz_a = [](int row) { return (row >> 1) & 5; };
  auto swz_b = [](int row) { return ((row >> 1) & 1) | (((row / (8 * FN)) & 1) << 2); };

  const int KB = (int)(g.k >> 7);
  const int ks0 = PARTIAL ? blockIdx.y * sps : 0;
  const int KS = PARTIAL ? min(sps, KB - ks0) : KB;
  // Direct loads: a uniform base and a 32-bit offset a lane (row pitches below
  // 2^24). Past the last stage they fetch it again, to a buffer nobody reads: no
  // branch in the loop.
  const uint8_t* sbase[LPW];
  uint32_t soff[LPW];
#pragma unroll
  for (int i = 0; i < LPW; ++i) {
    const int L = wave * LPW + i;
    if (L < BM / 8) {
      const int row = L * 8 + (lane >> 3), c = (lane & 7) ^ swz_a(row);
      sbase[i] = g.a + (int64_t)m0 * g.lda + (int64_t)ks0 * 128;
      soff[i] = (uint32_t)min(row, M - 1 - m0) * (uint32_t)g.lda + c * 16;
    } else {
      const int row = (L - BM / 8) * 8 + (lane >> 3), c = (lane & 7) ^ swz_b(row);
      sbase[i] = g.b + (int64_t)n0 * g.ldb + (int64_t)ks0 * 128;
      soff[i] = (uint32_t)min(row, N - 1 - n0) * (uint32_t)g.ldb + c * 16;
    }
  }
  // Scales, 64 to a load, one load a wave: those of a, then those of b's rows, or
  // of its blocks of 128 rows (surplus waves repeat one: the same bytes to the
  // same place).
  const int sl = wave < BM / 64 + (BROWS ? BN / 64 : 1) ? wave : wave % (BM / 64);
  const float* scbase = g.sa + (int64_t)ks0 * g.ldsa + m0;
  int64_t scoff = min(sl * 64 + lane, M - 1 - m0), scstep = g.ldsa;
  if (sl >= BM / 64) {
    scbase = BROWS ? g.sb + (int64_t)ks0 * g.ldsb + n0 : g.sb + (int64_t)(n0 >> 7) * g.ldsb + ks0;
    scoff = BROWS ? min((sl - BM / 64) * 64 + lane, N - 1 - n0)
                  : min(lane, min((BN - 1) >> 7, ((N - 1) >> 7) - (n0 >> 7))) * g.ldsb;
    scstep = BROWS ? g.ldsb : 1;
  }
  auto issue = [&](int ks) {
    uint8_t* const stage = ring + (ks & (NS - 1)) * Cfg::STAGE;
    const int at = min(ks, KS - 1);
#pragma unroll
    for (int i = 0; i < LPW; ++i)
      __builtin_amdgcn_global_load_lds((const void*)(sbase[i] + (int64_t)at * 128 + soff[i]),
                                       (lds_void_t*)(stage + (wave * LPW + i) * 1024), 16, 0, 0);
    __builtin_amdgcn_global_load_lds((const void*)(scbase + (int64_t)at * scstep + scoff),
                                     (lds_void_t*)(stage + Cfg::AB_BYTES + sl * 256), 4, 0, 0);
  };
  // Fragment addresses: the two granules of a lane differ by one bit.
  const int arow = wm0 + r16, brow = wn0 + 4 * FN * (r16 >> 2) + (r16 & 3);
  const int aoff = arow * 128 + (((2 * g4) ^ swz_a(arow)) << 4);  // (16 rows on: the same swizzle)
  const int boff = Cfg::A_BYTES + brow * 128 + (((2 * g4) ^ swz_b(brow)) << 4);  // (4 rows on: the same)
  auto read_a = [&](const uint8_t* st, int i) {
    const uint8_t* p = st + i * 2048;
    return join8(*reinterpret_cast<const u32x4_t*>(p + aoff), *reinterpret_cast<const u32x4_t*>(p + (aoff ^ 16)));
  };
  auto read_b = [&](const uint8_t* st, int j) {
    const uint8_t* p = st + j * 512;
    return join8(*reinterpret_cast<const u32x4_t*>(p + boff), *reinterpret_cast<const u32x4_t*>(p + (boff ^ 16)));
  };

  f32x4_t acc[FM][FN];

  constexpr int MFMAS = FN * (OUT_BF16 ? 1 : 4);
  constexpr int VALUS = (FN * (BROWS ? 8 : 4) + (OUT_BF16 ? 0 : 16) + MFMAS - 1) / MFMAS;
  // WIDE: with fold_wide. Otherwise reach says afterwards whether a scale may need it:
  // one that this wave fetched (FETCHED, a read of LDS a step), or the few that it
  // uses. The look at those it uses takes 2% of 300 x 4096 x 4096 (64 x 128 tiles,
  // 15.0 us) and 3% of 2000 x 4096 x 4096 (128 x 128, 38 us), at those it fetched 5%
  // and 1%.
  constexpr bool FETCHED = BROWS || FM > 2;
  uint32_t reach = 0;
  auto walk = [&](auto wide) {
    constexpr bool WIDE = decltype(wide)::value;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) issue(s);
    __builtin_amdgcn_s_waitcnt(VMCNT_ENCODE((NS - 2) * (LPW + 1)));
    barrier_only();
    for (int ks = 0; ks < KS; ++ks) {
      issue(ks + NS - 1);
      const uint8_t* st = ring + (ks & (NS - 1)) * Cfg::STAGE;
      const float* ss = reinterpret_cast<const float*>(st + Cfg::AB_BYTES);
      if constexpr (WIDE) {  // one fragment of b at a time: no more registers than the loop below
        const float sw = BROWS ? 1.f : ss[BM + (wn0 >> 7)];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          Frag<!OUT_BF16> wb[1], wa;
          wa.set(read_a(st, i));
          const float sa = ss[arow + 16 * i];
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            f32x4_t p[1];
            wb[0].set(read_b(st, j));
            block_sums(wb, wa, p);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i][j][e] = fold_wide(p[0][e], sa, BROWS ? ss[BM + wn0 + 4 * FN * g4 + 4 * j + e] : sw, acc[i][j][e]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      } else {
        Frag<!OUT_BF16> wb[FN], wa;
#pragma unroll
        for (int j = 0; j < FN; ++j) wb[j].set(read_b(st, j));
        i32x8_t fa = read_a(st, 0);
        const float sw = BROWS ? 1.f : ss[BM + (wn0 >> 7)];
        float sc[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) sc[i] = ss[arow + 16 * i];
        f32x4_t sbv[BROWS ? FN : 1];
        if constexpr (BROWS) {
#pragma unroll
          for (int j = 0; j < FN; ++j) sbv[j] = *reinterpret_cast<const f32x4_t*>(ss + BM + wn0 + 4 * FN * g4 + 4 * j);
        }
        float own = sw;
        f32x4_t p[2][FN];
        auto fold = [&](int i) {
          const float s = sc[i] * sw;
#pragma unroll
          for (int j = 0; j < FN; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i][j][e] = fmaf(p[i & 1][j][e], BROWS ? s * sbv[BROWS ? j : 0][e] : s, acc[i][j][e]);
            asm volatile("" : "+v"(acc[i][j]));  // here, not behind the barrier
          }
        };
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          wa.set(fa);
          if (i + 1 < FM) fa = read_a(st, i + 1);
          block_sums(wb, wa, p[i & 1]);
          if (FETCHED && i == FM - 2) own = ss[sl * 64 + lane];
          if (i > 0) fold(i - 1);
          if (i == (FETCHED ? FM - 1 : 0)) reach = max(reach, scale_reach(own, FETCHED && sl < BM / 64 ? A_BIAS : B_BIAS));
          if constexpr (!FETCHED) reach = max(reach, scale_reach(sc[i], A_BIAS));
#pragma unroll
          for (int t = 0; t < MFMAS; ++t) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, VALUS, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        fold(FM - 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(VMCNT_ENCODE((NS - 2) * (LPW + 1)) & LGKMCNT0_ENCODE);  // the next stage has landed
      barrier_only();
    }
    __builtin_amdgcn_s_waitcnt(VMCNT_ENCODE(0));  // no load to LDS outlives the block
  };
  walk(std::false_type{});
  // The sums again, with fp64 where it is needed, where a scale of the block is that
  // far from 1 (2.5 to 3 times the usual time; as a branch in the loop it spilled 258
  // registers of the largest tile).
  __shared__ uint32_t far_waves[Cfg::NW];
  const uint64_t far_lanes = __ballot(reach > MID_SCALES);  // (of all lanes: not inside the branch)
  if (lane == 0) far_waves[wave] = far_lanes != 0;
  __syncthreads();
  uint32_t any = 0;
#pragma unroll
  for (int w = 0; w < Cfg::NW; ++w) any |= far_waves[w];
  if (__builtin_amdgcn_readfirstlane(any) != 0) walk(std::true_type{});

  const int nb = n0 + wn0 + 4 * FN * g4;
  if constexpr (PARTIAL) {
    float* part = g.part + (int64_t)blockIdx.y * g.m * ldp;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = m0 + wm0 + i * 16 + r16;
      float v[4 * FN];
#pragma unroll
      for (int e = 0; e < 4 * FN; ++e) v[e] = acc[i][e >> 2][e & 3];
      if (row < M) store_cols<4 * FN>(part + (int64_t)row * ldp + nb, (int)ldp - nb, true, v);
    }
  } else {
    typedef typename std::conditional<OUT_BF16, uint16_t, float>::type out_t;
    const bool vec = (((uintptr_t)g.c | (uintptr_t)(g.ldc * (int64_t)sizeof(out_t))) & 15u) == 0;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = m0 + wm0 + i * 16 + r16;
      float v[4 * FN];
#pragma unroll
      for (int e = 0; e < 4 * FN; ++e) v[e] = acc[i][e >> 2][e & 3];
      if (row < M) store_cols<4 * FN>((out_t*)g.c + (int64_t)row * g.ldc + nb, N - nb, vec, v);
    }
  }
}

// The splits' sums, added in order.
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void k_qgemm_fp8_join(GemmFp8Args g, int splits, int64_t ldp) {
  typedef typename std::conditional<OUT_BF16, uint16_t, float>::type out_t;
  const int64_t quads = ldp / 4, total = g.m * quads;
  const bool vec = (((uintptr_t)g.c | (uintptr_t)(g.ldc * (int64_t)sizeof(out_t))) & 15u) == 0;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
    const int64_t row = t / quads, c = (t - row * quads) * 4;
    const float* p = g.part + row * ldp + c;
    f32x4_t s = *reinterpret_cast<const f32x4_t*>(p);
    for (int i = 1; i < splits; ++i) {
      const f32x4_t o = *reinterpret_cast<const f32x4_t*>(p + (int64_t)i * g.m * ldp);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += o[e];
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
    store_cols<4>((out_t*)g.c + row * g.ldc + c, (int)min((int64_t)4, g.n - c), vec, v);
  }
}

// Few rows: bound by the bytes of b, which go straight to registers (and are
// summed the exact way whatever C's type). A block takes 16 FN rows of b; its
// eight waves deal the steps of k among themselves, U of them in flight each, and
// join their sums through LDS in wave order. One row, n 4096, k 12288: 10.5 us, 50 MB
// of weights at 4.8 TB/s; 33 rows, n 1163, k 1280: 6.4 us (chains of loads).
template <int FM, int FN, int U, bool BROWS, bool OUT_BF16>
__global__ __launch_bounds__(512, 1) void k_qgemm_fp8_few(GemmFp8Args g) {
  constexpr int NW = 8;
  __shared__ f32x4_t sums[NW][FM * FN][64];
  const int n0 = blockIdx.x * 16 * FN;
  const int M = (int)g.m, N = (int)g.n, KB = (int)(g.k >> 7);
  const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint8_t *bp[FN], *ap[FM];
  const float* sp[FM];
#pragma unroll
  for (int j = 0; j < FN; ++j)
    bp[j] = g.b + (int64_t)min(n0 + 4 * FN * (r16 >> 2) + 4 * j + (r16 & 3), N - 1) * g.ldb + 32 * g4;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = min(16 * i + r16, M - 1);
    ap[i] = g.a + (int64_t)row * g.lda + 32 * g4;
    sp[i] = g.sa + row;
  }
  const int nb = n0 + 4 * FN * g4;
  const float* sbp = BROWS ? g.sb : g.sb + (int64_t)(n0 >> 7) * g.ldsb;
  f32x4_t acc[FM][FN];
  uint32_t reach = 0;  // of the scales that this wave meets, as in k_qgemm_fp8
  auto walk = [&](auto wide) {
    constexpr bool WIDE = decltype(wide)::value;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int ks0 = wave; ks0 < KB; ks0 += NW * U) {
      i32x8_t rb[U][FN], ra[U][FM];
      float sc[U][FM];
      f32x4_t sbv[U][FN];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // (past the last step: the last one again, with scales of zero)
        const int ks = ks0 + NW * u, at = min(ks, KB - 1);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const u32x4_t* p = reinterpret_cast<const u32x4_t*>(bp[j] + (int64_t)at * 128);
          rb[u][j] = join8(p[0], p[1]);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const u32x4_t* p = reinterpret_cast<const u32x4_t*>(ap[i] + (int64_t)at * 128);
          ra[u][i] = join8(p[0], p[1]);
          sc[u][i] = ks < KB ? sp[i][(int64_t)at * g.ldsa] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sbv[u][j][e] = BROWS ? sbp[(int64_t)at * g.ldsb + min(nb + 4 * j + e, N - 1)] : sbp[at];
      }
      __builtin_amdgcn_sched_barrier(0);  // all loads of the batch go out first
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u > 0 && ks0 + NW * u >= KB) break;
        if constexpr (!WIDE) {
#pragma unroll
          for (int i = 0; i < FM; ++i) reach = max(reach, scale_reach(sc[u][i], A_BIAS));
#pragma unroll
          for (int j = 0; j < (BROWS ? FN : 1); ++j)
#pragma unroll
            for (int e = 0; e < (BROWS ? 4 : 1); ++e) reach = max(reach, scale_reach(sbv[u][j][e], B_BIAS));
        }
        Frag<true> fb[FN], fa;
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j].set(rb[u][j]);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          fa.set(ra[u][i]);
          f32x4_t p[FN];
          block_sums(fb, fa, p);
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i][j][e] = WIDE ? fold_wide(p[j][e], sc[u][i], sbv[u][j][e], acc[i][j][e])
                                  : fmaf(p[j][e], sc[u][i] * sbv[u][j][e], acc[i][j][e]);
        }
      }
    }
  };
  walk(std::false_type{});
  if (__ballot(reach > MID_SCALES) != 0) walk(std::true_type{});
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) sums[wave][i * FN + j][lane] = acc[i][j];
  __syncthreads();
  typedef typename std::conditional<OUT_BF16, uint16_t, float>::type out_t;
  const bool vec = (((uintptr_t)g.c | (uintptr_t)(g.ldc * (int64_t)sizeof(out_t))) & 15u) == 0;
  for (int t = threadIdx.x; t < FM * FN * 64; t += 512) {
    const int f = t >> 6, l = t & 63, row = 16 * (f / FN) + (l & 15);
    const int c = n0 + 4 * FN * (l >> 4) + 4 * (f % FN);
    f32x4_t s = sums[0][f][l];
#pragma unroll
    for (int w = 1; w < NW; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += sums[w][f][l][e];
    const float v[4] = {s.x, s.y, s.z, s.w};
    if (row < M) store_cols<4>((out_t*)g.c + (int64_t)row * g.ldc + c, N - c, vec, v);
  }
}

// ---------------------------------------------------------------- launchers
namespace {

constexpr int64_t F8_CUS = 256;

enum F8Tile { F8_FEW, F8_256x256, F8_128x128, F8_64x128 };
struct F8Plan {
  F8Tile tile;
  int splits, sps;
};

int64_t tiles_of(int64_t m, int64_t n, int64_t bm, int64_t bn) { return ((m + bm - 1) / bm) * ((n + bn - 1) / bn); }

// The tile and the splits of k that take the least time by these measured times
// of a step of k (bf16 C, fp32 C):
//   64 x 128    four stages, a block a compute unit: 0.42, 0.8 us
//   128 x 128   two stages, two blocks a compute unit: 1.13, 2.8 us for both of
//               them, 0.72, 1.4 for one that is alone (2.8 with a scale a row of b;
//               with its blocks 2.1, which the rule does not tell apart: 1200 x 4096
//               x 4096 takes 64 x 128 and 76 us, where 2.1 would give 67)
//   256 x 256   two stages, a block a compute unit, bf16 C only (the widened
//               fragments do not fit beside its sums): 2.05 us
// and of a split product's join, 3 us and a write and a read of the partial sums
// at 3 TB/s. Measured: 2000 x 4096, k 4096, bf16, 128 x 128 39 us, 256 x 256 57;
// 4096 x 12288 the same way 232 and 200; 300 x 4096, 64 x 128 15.5 us, 128 x 128
// 24; 64 x 4096, k 12288, 64 x 128 37 us unsplit, 15.6 in 6 splits.
// Few rows: one block row of 16 takes their bytes of b once more each, so up to
// 16 rows always, up to 64 where 16-row blocks times n k stay below 2^25 (32 x
// 4096 x 4096 9.1 against 11.4 us, 64 x 4096 x 4096 14.4 against 11.4).
F8Plan plan_of(int64_t m, int64_t n, int64_t k, bool c_bf16) {
  const int64_t kb = k / 128;
  if (m <= 16 || (m <= 64 && (m + 15) / 16 * n * k <= ((int64_t)1 << 25))) return F8Plan{F8_FEW, 1, 0};
  const double step64 = c_bf16 ? 0.42 : 0.8, one128 = c_bf16 ? 0.72 : 1.4, two128 = c_bf16 ? 1.13 : 2.8;
  auto rounds = [](int64_t tiles) { return (tiles + F8_CUS - 1) / F8_CUS; };
  const int64_t t64 = tiles_of(m, n, 64, 128), r128 = rounds(tiles_of(m, n, 128, 128));
  F8Plan best{F8_128x128, 1, (int)kb};
  double least = ((double)(r128 / 2) * two128 + (double)(r128 & 1) * one128) * (double)kb;
  const double big = (double)rounds(tiles_of(m, n, 256, 256)) * 2.05 * (double)kb;
  if (c_bf16 && big < least) {
    best = F8Plan{F8_256x256, 1, (int)kb};
    least = big;
  }
  for (int64_t s = 1; s <= kb && s <= 16 && (s == 1 || (t64 * s <= F8_CUS)); ++s) {
    const int64_t sps = (kb + s - 1) / s, splits = (kb + sps - 1) / sps;
    const double join = splits == 1 ? 0.0 : 3.0 + (double)(splits * m * n) * 8.0 / 3e6;
    const double t = (double)rounds(t64 * splits) * (double)sps * step64 + join;
    if (t < least) {
      best = F8Plan{F8_64x128, (int)splits, (int)sps};
      least = t;
    }
  }
  return best;
}

int64_t pitch_of(int64_t n) { return (n + 3) / 4 * 4; }

// gm: tile rows that an XCD walks together (pp_map_tile).
template <int BM, int BN, int WM, int WN, int NS, bool BROWS, bool OUT_BF16>
hipError_t tile_launch(const GemmFp8Args& g, const F8Plan& p, int gm, hipStream_t stream) {
  using Cfg = F8Cfg<BM, BN, WM, WN, NS>;
  const int tiles_m = (int)((g.m + BM - 1) / BM), tiles_n = (int)((g.n + BN - 1) / BN);
  const dim3 grid((unsigned)(tiles_m * tiles_n), (unsigned)p.splits), block(Cfg::NT);
  const int64_t ldp = pitch_of(g.n);
  if (p.splits == 1) {
    hipLaunchKernelGGL((k_qgemm_fp8<BM, BN, WM, WN, NS, BROWS, OUT_BF16, false>), grid, block, Cfg::LDS_BYTES, stream,
                       g, tiles_m, tiles_n, gm, p.sps, ldp);
    return hipGetLastError();
  }
  if constexpr (BM == 64) {  // (plan_of splits nothing else)
    if (g.part == nullptr) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_qgemm_fp8<BM, BN, WM, WN, NS, BROWS, OUT_BF16, true>), grid, block, Cfg::LDS_BYTES, stream,
                       g, tiles_m, tiles_n, gm, p.sps, ldp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = std::min<int64_t>((g.m * (ldp / 4) + 255) / 256, 65536);
    hipLaunchKernelGGL((k_qgemm_fp8_join<OUT_BF16>), dim3((unsigned)blocks), dim3(256), 0, stream, g, p.splits, ldp);
    return hipGetLastError();
  }
  return hipErrorInvalidValue;
}

template <int FM, int U, bool BROWS>
hipError_t few_launch(const GemmFp8Args& g, hipStream_t stream) {
  constexpr int FN = 1;
  const dim3 grid((unsigned)((g.n + 16 * FN - 1) / (16 * FN))), block(512);
  if (g.c_bf16)
    hipLaunchKernelGGL((k_qgemm_fp8_few<FM, FN, U, BROWS, true>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((k_qgemm_fp8_few<FM, FN, U, BROWS, false>), grid, block, 0, stream, g);
  return hipGetLastError();
}

template <bool BROWS, bool OUT_BF16>
hipError_t plan_launch(const GemmFp8Args& g, const F8Plan& p, hipStream_t stream) {
  switch (p.tile) {
    case F8_FEW:
      if (g.m <= 16) return few_launch<1, 4, BROWS>(g, stream);
      if (g.m <= 32) return few_launch<2, 2, BROWS>(g, stream);
      return few_launch<4, 2, BROWS>(g, stream);
    case F8_256x256:
      if constexpr (OUT_BF16) return tile_launch<256, 256, 128, 64, 2, BROWS, true>(g, p, 8, stream);
      break;
    case F8_128x128: return tile_launch<128, 128, 64, 64, 2, BROWS, OUT_BF16>(g, p, 8, stream);
    case F8_64x128: return tile_launch<64, 128, 32, 32, 4, BROWS, OUT_BF16>(g, p, 8, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

int64_t qgemm_fp8_partial_bytes(int64_t m, int64_t n, int64_t k, bool c_bf16) {
  const F8Plan p = plan_of(m, n, k, c_bf16);
  return p.splits == 1 ? 0 : (int64_t)p.splits * m * pitch_of(n) * 4;
}

hipError_t launch_qgemm_fp8(const GemmFp8Args& g, hipStream_t stream) {
  const F8Plan p = plan_of(g.m, g.n, g.k, g.c_bf16);
  if (g.b_rows) return g.c_bf16 ? plan_launch<true, true>(g, p, stream) : plan_launch<true, false>(g, p, stream);
  return g.c_bf16 ? plan_launch<false, true>(g, p, stream) : plan_launch<false, false>(g, p, stream);
}

}  // namespace tp
