// Dropout of a branch, residual addition, layer norm and rotation of whole rows
// in front of a projection, and their gradients.
//
//   t  = stream(drop(x) + residual), or x
//   mu = mean(t)      r = (mean((t - mu)^2) + eps)^(-1/2)
//   h  = (t - mu) r gamma + beta             h' = h . blockdiag(H / 16)
//
// The row sits in the registers of its sets of lanes (row_sets.hpp), so the
// mean comes first and the squares are those of the deviations: no digits are
// lost in rows far off zero, and every element is read once.
#include <algorithm>
#include <type_traits>

#include "block_ops.hpp"
#include "e4m3.hpp"
#include "lanes.hpp"
#include "philox.hpp"
#include "row_sets.hpp"

namespace tp {

enum { LN_OUT_I8 = 0, LN_OUT_BF16 = 1, LN_OUT_FP8 = 2 };

// Sums (or maxima) of N values over the threads of a row: all threads of the block
// call it, with red [N][JOIN] of its own for each join of a row. Where a block
// has one wide row its waves' results are met all at once (red holds zeros past
// the last wave); rows that share a block (of up to three sets forward, of up to
// eight in the gradients) are met set by set.
constexpr int JOIN = 16;  // results of a join: the most waves, and the sets of a block of short rows

template <int N, bool MAX, int WAVES>
__device__ __forceinline__ void row_join(double (&v)[N], const Place& pl, int groups, double* red) {
  __builtin_amdgcn_sched_barrier(0);  // nothing of the next phase before this one: registers
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = row_all<MAX>(v[i]);
  if (WAVES > 4 || pl.wide) {  // sets past the row hold zeros
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = rows_all<MAX>(v[i]);
      if ((threadIdx.x & 63) == 0) red[i * JOIN + (threadIdx.x >> 6)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0;
#pragma unroll
      for (int q = 0; q < WAVES; q += 4) {  // four at a time: fewer registers
        const double2 e = *reinterpret_cast<const double2*>(red + i * JOIN + q);
        const double2 f = *reinterpret_cast<const double2*>(red + i * JOIN + q + 2);
        v[i] = meet<MAX>(v[i], meet<MAX>(meet<MAX>(e.x, e.y), meet<MAX>(f.x, f.y)));
        asm volatile("" : "+v"(v[i]));  // summed here
      }
    }
  } else {  // (16 sets at most)
    if (pl.l16 == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * JOIN + pl.set] = v[i];
    }
    __syncthreads();
    const int first = pl.slot * groups, count = pl.active ? groups : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0;
      for (int w = 0; w < count; ++w) v[i] = meet<MAX>(v[i], red[i * JOIN + first + w]);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
}

// The eight dwords of a lane's 16 bf16 weights; fp32 ones are fetched where they
// are used.
struct Weights16 {
  u32x4_t w[2];
  __device__ __forceinline__ void fetch(const VecArg& g, bool bf16, int64_t c, uint32_t none) {
    w[0] = w[1] = u32x4_t{none, none, none, none};
    if (g.p != nullptr && bf16) {
      w[0] = *reinterpret_cast<const u32x4_t*>((const uint16_t*)g.p + c);
      w[1] = *reinterpret_cast<const u32x4_t*>((const uint16_t*)g.p + c + 128);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t v = w[i >> 3][(i >> 1) & 3];
    return (i & 1) ? bf16_hi(v) : bf16_lo(v);
  }
};

// sum / k with its remainder taken back: the mean of equal values is that value,
// so a constant row has deviations of zero.
__device__ __forceinline__ double row_mean(double sum, double k, double inv_k) {
  const double q = sum * inv_k;
  return fma(fma(-q, k, sum), inv_k, q);
}

// What is read again after a join is widened again: not kept in twice the
// registers across it.
template <int N>
__device__ __forceinline__ void afresh(float (&t)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(t[i]));
}

// ------------------------------------------------------------------ forward
// Codes: fp64 throughout, so they are those of exact arithmetic on the normed
// row. bf16 rows: the row's sums in fp64, the rest in fp32, one rounding; a
// deviation is the difference from the mean's two fp32 parts, as exact as t
// allows. bf16 weights are fetched with the row.
//
// A block has one row (or a few short ones) and walks none: 72 to 96 registers
// instead of the 128 of a loop with its addresses and weights (4096 x 4096, bf16 and
// its stream, dropout, rotated bf16 rows: 33.5 -> 26.5 us, with the sums across lanes
// on the vector unit).
// bf16 rows are bound by HBM (those 26.5 us: 5.1 TB/s), codes by fp64 beside it
// (e4m3 codes of 2000 x 8192, fp32 in, bf16 stream: 33.1 us, 4.5 TB/s; int8 codes with
// their third join 36.7, 4.0 TB/s, rotated 39, and of 4096 x 4096 in bf16 with the
// dropout, rotated, 38, 3.1 TB/s), one row of 4096 by its chain of three joins (4.3).
template <typename TX, typename TS, bool RES, int OUT, int NT>
__global__ __launch_bounds__(NT, 4) void k_layernorm(LayerNormArgs a, int rows_per_block, int64_t row0) {
  typedef typename std::conditional<OUT == LN_OUT_BF16, float, double>::type T;
  constexpr int SET_BYTES = 16 * (16 + (sizeof(T) == 4 ? 4 : 2)) * (int)sizeof(T);
  extern __shared__ __align__(16) uint8_t lds[];
  const Place pl = place_of(a.groups, rows_per_block);
  uint8_t* bbuf = lds + pl.set * SET_BYTES;
  T* tbuf = reinterpret_cast<T*>(bbuf);
  constexpr int WAVES = NT / 64;
  double* red = reinterpret_cast<double*>(lds + (blockDim.x >> 4) * SET_BYTES);  // [3][JOIN]
  const uint32_t col = pl.grp * 256 + pl.l16 * 8;
  const int64_t k = (int64_t)a.groups * 256;
  const double inv_k = 1.0 / (double)k;
  const bool wb = a.gamma.p != nullptr ? a.gamma.bf16 : a.beta.bf16;
  if (threadIdx.x < 3 * JOIN) red[threadIdx.x] = 0.0;
  __syncthreads();
  // (a wide row is the whole block's: its addresses take no registers of the lanes)
  const int64_t row = row0 + (NT > 256 ? blockIdx.x : blockIdx.x * (int64_t)pl.rows + pl.slot);
  const bool live = pl.active && row < a.m;
  Runs<TX> rx;
  Runs<TS> rr;
  Weights16 gw, bw;
  gw.fetch(a.gamma, pl.active && wb, col, 0x3f803f80u);
  bw.fetch(a.beta, pl.active && wb, col, 0u);
  if (live) {
    rx.load((const TX*)a.x + row * a.ldx + col);
    if constexpr (RES) rr.load((const TS*)a.res + row * a.ldr + col);
  } else {
    rx.zero();
    if constexpr (RES) rr.zero();
  }
  float t[16];
  if (RES && a.drop.rng != nullptr) {
    const PhiloxKey key = philox_key(a.drop.rng);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4_t w = philox4x32_10(key, (uint64_t)(row * k + col + 128 * h) >> 3);
#pragma unroll
      for (int j = 0; j < 8; ++j) t[8 * h + j] = philox_drop(w, j, a.drop, rx.get(8 * h + j));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = rx.get(i);
  }
  if constexpr (RES) {
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = as_stream<TS>(t[i] + rr.get(i));
    if (live) store16((TS*)a.sum + row * a.ldsum + col, t);
  }

  double s[1] = {0.0};
#pragma unroll
  for (int i = 0; i < 16; ++i) s[0] += (double)t[i];
  row_join<1, false, WAVES>(s, pl, a.groups, red);
  const double mu = row_mean(s[0], (double)k, inv_k);
  const float mu_hi = (float)mu, mu_lo = (float)(mu - (double)mu_hi);
  if (OUT != LN_OUT_BF16) afresh(t);
  s[0] = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (OUT == LN_OUT_BF16) {
      t[i] = (t[i] - mu_hi) - mu_lo;
      s[0] = fma((double)t[i], (double)t[i], s[0]);
    } else {
      const double d = (double)t[i] - mu;
      s[0] = fma(d, d, s[0]);
    }
  }
  if (!pl.active) s[0] = 0.0;
  row_join<1, false, WAVES>(s, pl, a.groups, red + JOIN);
  const double r = 1.0 / sqrt(s[0] * inv_k + a.eps);
  if (OUT != LN_OUT_BF16) afresh(t);

  T v[16];
  auto apply = [&](int i, float gm, float bt) {
    if constexpr (OUT == LN_OUT_BF16)
      v[i] = fmaf(t[i] * (float)r, gm, bt);
    else
      v[i] = fma(((double)t[i] - mu) * r, (double)gm, (double)bt);
  };
  if (wb || (a.gamma.p == nullptr && a.beta.p == nullptr)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      apply(i, gw.get(i), bw.get(i));
      if (OUT != LN_OUT_BF16 && (i & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // four at a time: fewer registers
    }
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      f32x4_t gm = {1.f, 1.f, 1.f, 1.f}, bt = {0.f, 0.f, 0.f, 0.f};
      const int64_t c = col + 128 * (h >> 1) + 4 * (h & 1);
      if (pl.active && a.gamma.p != nullptr) gm = *reinterpret_cast<const f32x4_t*>((const float*)a.gamma.p + c);
      if (pl.active && a.beta.p != nullptr) bt = *reinterpret_cast<const f32x4_t*>((const float*)a.beta.p + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) apply(4 * h + e, gm[e], bt[e]);
    }
  }
  if (!pl.active) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0;
  }
  if (a.rotate) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= (T)0.0625;
    fwht16_regs(v);
    transpose16(v, tbuf, pl.l16);
    fwht16_regs(v);
  } else if (OUT == LN_OUT_I8) {
    transpose16(v, tbuf, pl.l16);  // the same output order either way
  }
  // after the transpose register q is element l16 of lane q's two runs
  const int at = 128 * (pl.l16 >> 3) + (pl.l16 & 7);

  if constexpr (OUT == LN_OUT_BF16) {
    if (a.rotate) transpose16_back(v, tbuf, pl.l16);
    if (live) store16((uint16_t*)a.y + row * a.ldy + col, v);
  } else if constexpr (OUT == LN_OUT_FP8) {
    // A set holds two blocks of 128: after the transform its lanes 0 .. 7 hold
    // the first one, without it the first run of every lane is the first one's.
    uint8_t* yrow = (uint8_t*)a.y + row * a.ldy + (int64_t)pl.grp * 256;
    if (a.rotate) {
      double am = absmax16(v);
      am = fmax(am, swz_xor<1>(am));
      am = fmax(am, swz_xor<2>(am));
      am = fmax(am, swz_xor<4>(am));
      const float sc = e4m3_scale(am);
      const E4m3Inverse inv = e4m3_inverse(sc);
      uint32_t w[4];
      e4m3_codes<16>(w, [&](int i) { return (float)v[i]; }, [&](int i) { return v[i]; }, [&](int) { return inv; },
                       inv.slow());
      wave_lds_sync();
#pragma unroll
      for (int q = 0; q < 16; ++q) bbuf[at + 8 * q] = (uint8_t)(w[q >> 2] >> (8 * (q & 3)));
      wave_lds_sync();
      const u32x4_t w4 = *reinterpret_cast<const u32x4_t*>(bbuf + 16 * pl.l16);
      if (live) {
        *reinterpret_cast<u32x4_t*>(yrow + 16 * pl.l16) = w4;
        if ((pl.l16 & 7) == 0) a.scales[(2 * pl.grp + (pl.l16 >> 3)) * a.ldscales + row] = sc;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        double am = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) am = absmax2(am, v[8 * h + j]);
        const float sc = e4m3_scale(row_all<true>(am));
        const E4m3Inverse inv = e4m3_inverse(sc);
        uint32_t w2[2];
        e4m3_codes<8>(w2, [&](int i) { return (float)v[8 * h + i]; }, [&](int i) { return v[8 * h + i]; },
                      [&](int) { return inv; }, inv.slow());
        if (live) {
          *reinterpret_cast<uint2*>(yrow + 128 * h + 8 * pl.l16) = uint2{w2[0], w2[1]};
          if (pl.l16 == 0) a.scales[(2 * pl.grp + h) * a.ldscales + row] = sc;
        }
      }
    }
  } else {
    // Maxima drop NaN: a row that holds one gets an infinite scale, so that what reads
    // it is not finite either. (A rotated group is NaN everywhere.)
    uint32_t top = (uint32_t)(__builtin_bit_cast(uint64_t, v[0]) >> 32) & 0x7fffffffu;
    if (!a.rotate) {
#pragma unroll
      for (int i = 1; i < 16; ++i) top = max(top, (uint32_t)(__builtin_bit_cast(uint64_t, v[i]) >> 32) & 0x7fffffffu);
    }
    double am[1] = {top > 0x7ff00000u ? __builtin_inf() : absmax16(v)};
    row_join<1, true, WAVES>(am, pl, a.groups, red + 2 * JOIN);
    const float s32 = (float)(am[0] / 127.0);
    const double s64 = (double)s32, inv64 = s32 > 0.f ? 1.0 / s64 : 0.0;
    constexpr double MAGIC = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer (RNE)
    // The product with 1 / s decides the code unless it is within 1e-9 of a tie;
    // rows with a subnormal scale take the division.
    const bool direct = s32 == 0.f || s32 >= 0x1p-126f;
    wave_lds_sync();
    bool tie = false;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const double f = fma(v[q], inv64, MAGIC);
      const double d = fma(v[q], inv64, MAGIC - f);
      tie |= !(fabs(d) < 0.5 - 1e-9);
      bbuf[at + 8 * q] = (uint8_t)__builtin_bit_cast(uint64_t, f);
      if ((q & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // four codes at a time: fewer registers
    }
    if (__ballot((tie || !direct) && live)) {
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const double f = fma(v[q], inv64, MAGIC);
        const double d = fma(v[q], inv64, MAGIC - f);
        if (!direct || !(fabs(d) < 0.5 - 1e-9)) bbuf[at + 8 * q] = (uint8_t)quant_code(v[q], s64, inv64, 127.0);
        __builtin_amdgcn_sched_barrier(0);  // one division at a time
      }
    }
    wave_lds_sync();
    const u32x4_t w4 = *reinterpret_cast<const u32x4_t*>(bbuf + 16 * pl.l16);
    if (live) {
      *reinterpret_cast<u32x4_t*>((uint8_t*)a.y + row * a.ldy + (int64_t)pl.grp * 256 + 16 * pl.l16) = w4;
      if (pl.grp == 0 && pl.l16 == 0) a.scales[row] = s32;
    }
  }
}

// ----------------------------------------------------------------- backward
//   g = dy . blockdiag(H / 16) (the rotation is its own inverse), or dy
//   n = (t - mu) r;  w = gamma g
//   dt = r (w - mean(w) - n mean(w n)) + dsum;   dbranch = drop(dt)
//   dgamma = sum over rows of g n;               dbeta = sum over rows of g
// fp32, the row's sums in fp64; a deviation is the difference from the mean's two
// fp32 parts.
//
// SUMS: a thread keeps its 16 columns of dgamma and dbeta over the rows of its
// block; the blocks' sums are joined by k_colsum in a fixed order. Wide rows
// (more than 16 groups) have no registers for that, and as many blocks as rows:
// their kernel leaves mu and r of each row, and k_layernorm_dw takes the sums.
// Measured: 4096 x 4096, fp32 dy, bf16 t, dsum and dx, with the dropout 45.1 us
// (HBM: 201 MB, 4.4 TB/s, three waves a SIMD: four spilled and were slower) and
// 4.4 for the join of 512 partial rows; 333 x 12288 fp32 15.7 us (1.3 rows a
// compute unit, each a chain of two joins), 7.0 for the sums' kernel (dy and t
// again, from the last-level cache) and 1.9 (minima of a trace; 50.8 and 5.1, 16.2,
// 7.8 and 3.0 at the median).
template <typename T>
__device__ __forceinline__ void rotate_back(float (&g)[16], const Runs<T>& raw, float* buf, int l16) {
#pragma unroll
  for (int i = 0; i < 16; ++i) g[i] = raw.get(i) * 0.0625f;
  fwht16_regs(g);
  transpose16(g, buf, l16);
  fwht16_regs(g);
  transpose16_back(g, buf, l16);
}

// Waves of a SIMD that the registers are cut for. Wide rows: six (80 registers)
// where dx and gamma are bf16, five else, which spilled 7 to 27 of 80 (all fp32,
// dsum, rotated: 2048 x 8192 101 -> 80 us, 2000 x 4352 62 -> 47; 333 x 12288 with an
// fp32 gamma 29.5 -> 26.5).
constexpr int ln_bwd_waves(bool dx_bf16, bool gamma_bf16, bool sums) {
  return sums ? 3 : dx_bf16 && gamma_bf16 ? 6 : 5;
}

template <typename TG, typename TT, typename TD, bool WB, int NT, bool SUMS>
__global__ __launch_bounds__(NT, ln_bwd_waves(sizeof(TD) == 2, WB, SUMS)) void k_layernorm_bwd(LayerNormBwdArgs a,
                                                                                            int rows_per_block,
                                                                                            int64_t row0) {
  constexpr int SET_BYTES = 16 * (16 + 4) * 4;
  extern __shared__ __align__(16) uint8_t lds[];
  const Place pl = place_of(a.groups, rows_per_block);
  float* tbuf = reinterpret_cast<float*>(lds + pl.set * SET_BYTES);
  constexpr int WAVES = NT / 64;
  double* red = reinterpret_cast<double*>(lds + (blockDim.x >> 4) * SET_BYTES);  // [4][JOIN]
  if (threadIdx.x < 4 * JOIN) red[threadIdx.x] = 0.0;
  __syncthreads();
  const uint32_t col = pl.grp * 256 + pl.l16 * 8;
  const int64_t k = (int64_t)a.groups * 256;
  const double inv_k = 1.0 / (double)k;

  // gamma: bf16 (or ones) as it lies in memory, or fp32
  Weights16 gw;
  float gf[WB ? 1 : 16], dg[16], db[16];
  if constexpr (WB) {
    gw.fetch(a.gamma, pl.active, col, pl.active ? 0x3f803f80u : 0u);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) gf[i] = 0.f;
    if (pl.active) load_vec16(a.gamma, col, gf);
  }
  auto gm = [&](int i) { return WB ? gw.get(i) : gf[WB ? 0 : i]; };
#pragma unroll
  for (int i = 0; i < 16; ++i) dg[i] = db[i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * pl.rows;
  for (int64_t base = row0 + (int64_t)blockIdx.x * pl.rows; base < a.m; base += step) {
    const int64_t row = SUMS ? base + pl.slot : base;
    const bool live = pl.active && row < a.m;
    Runs<TG> rg;
    Runs<TT> rt;
    Runs<TD> rd;
    rd.zero();
    if (live) {
      rt.load((const TT*)a.t + row * a.ldt + col);
      rg.load((const TG*)a.dy + row * a.lddy + col);
      if (a.dsum != nullptr) rd.load((const TD*)a.dsum + row * a.ldds + col);
    } else {
      rg.zero();
      rt.zero();
    }
    __builtin_amdgcn_sched_barrier(0);
    double c[3] = {0.0, 0.0, 0.0}, mean[1] = {0.0};
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      t[i] = rt.get(i);
      mean[0] += (double)t[i];
    }
    row_join<1, false, WAVES>(mean, pl, a.groups, red);
    __builtin_amdgcn_sched_barrier(0);
    const double mu = row_mean(mean[0], (double)k, inv_k);
    const float mu_hi = (float)mu, mu_lo = (float)(mu - (double)mu_hi);
    float g[16];
    if (a.rotate) {
      rotate_back(g, rg, tbuf, pl.l16);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) g[i] = rg.get(i);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      t[i] = (t[i] - mu_hi) - mu_lo;  // the deviation
      if (!SUMS) g[i] *= gm(i);  // (g itself is not used again)
      const double d = (double)t[i], w = (double)(SUMS ? g[i] * gm(i) : g[i]);
      c[0] += w;
      c[1] = fma(w, d, c[1]);
      c[2] = fma(d, d, c[2]);
      if ((i & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // four at a time: fewer registers
    }
    __builtin_amdgcn_sched_barrier(0);
    if (!pl.active) c[2] = 0.0;
    row_join<3, false, WAVES>(c, pl, a.groups, red + JOIN);
    const double r64 = 1.0 / sqrt(c[2] * inv_k + a.eps);
    const float r = (float)r64, m1 = (float)(c[0] * inv_k), m2 = (float)(r64 * (c[1] * inv_k));
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float n = t[i] * r;
      o[i] = fmaf(r, fmaf(-n, m2, (SUMS ? g[i] * gm(i) : g[i]) - m1), rd.get(i));
      if constexpr (SUMS) {
        if (live) {
          dg[i] = fmaf(g[i], n, dg[i]);
          db[i] += g[i];
        }
      }
      if ((i & 3) == 3) __builtin_amdgcn_sched_barrier(0);
    }
    if (live) {
      if (!SUMS && a.stats != nullptr && pl.grp == 0 && pl.l16 == 0)
        reinterpret_cast<double2*>(a.stats)[row] = double2{mu, r64};
      store16((TD*)a.dx + row * a.lddx + col, o);
      if (a.dbranch != nullptr) {
        __builtin_amdgcn_sched_barrier(0);  // the generator's registers come last
        if (a.drop.rng != nullptr) {
          const PhiloxKey key = philox_key(a.drop.rng);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4_t w = philox4x32_10(key, (uint64_t)(row * k + col + 128 * h) >> 3);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[8 * h + j] = philox_drop(w, j, a.drop, o[8 * h + j]);
          }
        }
        store16((TD*)a.dbranch + row * a.lddb + col, o);
      }
    }
    if (!SUMS) return;  // (one row a block)
  }
  if (!SUMS || (a.dgamma == nullptr && a.dbeta == nullptr)) return;
  float* part = a.part + (int64_t)blockIdx.x * (2 * k);
  if (pl.rows == 1) {
    if (pl.active) {
      store16(part + col, dg);
      store16(part + k + col, db);
    }
    return;
  }
  // the sums of the block's rows, added in order
  float* sums = reinterpret_cast<float*>(lds);  // [rows][columns]: 1 KiB of a set's 1.25 KiB
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    if (pl.active) store16(sums + pl.slot * k + col, which ? db : dg);
    __syncthreads();
    for (int c = threadIdx.x; c < (int)k; c += (int)blockDim.x) {
      float s = sums[c];
      for (int w = 1; w < pl.rows; ++w) s += sums[w * k + c];
      part[which * k + c] = s;
    }
  }
}

// dgamma and dbeta of wide rows: a block takes 256 columns of a share of the
// rows, its 16 sets a row each in turn; the sets' sums are added in order.
template <typename TG, typename TT>
__global__ __launch_bounds__(256) void k_layernorm_dw(LayerNormBwdArgs a, int shares) {
  constexpr int SET_BYTES = 16 * (16 + 4) * 4;
  __shared__ __align__(16) uint8_t lds[16 * SET_BYTES];
  const int l16 = threadIdx.x & 15, set = threadIdx.x >> 4;
  const int share = blockIdx.x / a.groups, grp = blockIdx.x - share * a.groups;
  const int64_t col = (int64_t)grp * 256 + l16 * 8, k = (int64_t)a.groups * 256;
  const int64_t r0 = a.m * share / shares, r1 = a.m * (share + 1) / shares;
  float dg[16], db[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dg[i] = db[i] = 0.f;
  for (int64_t row = r0 + set; row < r1; row += 16) {
    Runs<TG> rg;
    Runs<TT> rt;
    rg.load((const TG*)a.dy + row * a.lddy + col);
    rt.load((const TT*)a.t + row * a.ldt + col);
    const double2 st = reinterpret_cast<const double2*>(a.stats)[row];
    const float mu_hi = (float)st.x, mu_lo = (float)(st.x - (double)mu_hi), r = (float)st.y;
    float g[16];
    if (a.rotate) {
      rotate_back(g, rg, reinterpret_cast<float*>(lds + set * SET_BYTES), l16);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) g[i] = rg.get(i);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      dg[i] = fmaf(g[i], ((rt.get(i) - mu_hi) - mu_lo) * r, dg[i]);
      db[i] += g[i];
    }
  }
  float* sums = reinterpret_cast<float*>(lds);  // [16][256]
  float* part = a.part + (int64_t)share * (2 * k) + (int64_t)grp * 256;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    store16(sums + set * 256 + 8 * l16, which ? db : dg);
    __syncthreads();
    float s = sums[threadIdx.x];
#pragma unroll
    for (int w = 1; w < 16; ++w) s += sums[w * 256 + threadIdx.x];
    part[which * k + threadIdx.x] = s;
  }
}

// ---------------------------------------------------------------- launchers
namespace {

constexpr int64_t LN_BLOCKS = 1 << 21;  // of a launch, whose threads are counted in 32 bits
// Partial rows of dgamma and dbeta, a pass at 512, 256 and 1024 blocks: 4096 x 4096,
// fp32 dy and dropout 55.4, 68.5 and 58.5 us; 16384 x 1024 bf16 37.7, 51.9 and 40.5;
// 4096 x 2048 bf16 25.6, 32.2 and 28.6.
constexpr int64_t LN_BWD_BLOCKS = 512;
// Rows of more groups leave their sums to k_layernorm_dw (a thread of 16 groups'
// block keeps its 32 sums). A pass of 16 groups with the sums kept and left: 4096 x
// 4096, fp32 dy and dropout 55.4 and 69.5 us, bf16 38.6 and 40.0; 300 x 4096 fp32
// 15.5 and 19.2.
constexpr int LN_WIDE_GROUPS = 16;

template <typename TX, typename TS, bool RES, int OUT>
hipError_t ln_launch(const LayerNormArgs& a, hipStream_t stream) {
  const Shape s = shape_of(a.m, a.groups, LN_BLOCKS);
  const int set_bytes = OUT == LN_OUT_BF16 ? 16 * 20 * 4 : 16 * 18 * 8;
  const size_t lds = (size_t)(s.threads / 16) * set_bytes + 3 * JOIN * sizeof(double);
  for (int64_t row0 = 0; row0 < a.m; row0 += s.blocks * s.rows) {
    const int64_t blocks = std::min(s.blocks, (a.m - row0 + s.rows - 1) / s.rows);
    const dim3 grid((unsigned)blocks), block((unsigned)s.threads);
    if (s.threads <= 256)
      hipLaunchKernelGGL((k_layernorm<TX, TS, RES, OUT, 256>), grid, block, lds, stream, a, s.rows, row0);
    else
      hipLaunchKernelGGL((k_layernorm<TX, TS, RES, OUT, 1024>), grid, block, lds, stream, a, s.rows, row0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename TX, typename TS, bool RES>
hipError_t ln_out(const LayerNormArgs& a, hipStream_t stream) {
  if (a.out == LN_OUT_I8) return ln_launch<TX, TS, RES, LN_OUT_I8>(a, stream);
  if (a.out == LN_OUT_BF16) return ln_launch<TX, TS, RES, LN_OUT_BF16>(a, stream);
  return ln_launch<TX, TS, RES, LN_OUT_FP8>(a, stream);
}

template <typename TX>
hipError_t ln_x(const LayerNormArgs& a, hipStream_t stream) {
  if (a.res == nullptr) return ln_out<TX, float, false>(a, stream);
  return a.s_bf16 ? ln_out<TX, uint16_t, true>(a, stream) : ln_out<TX, float, true>(a, stream);
}

// Rows that keep their sums share a block of 16 sets, as long as 256 blocks have
// work (one row a block from four groups on: 16384 x 1024 69.5 against 37.7 us,
// 4096 x 2048 31.2 against 25.6).
Shape ln_bwd_shape(int64_t m, int groups) {
  if (groups > LN_WIDE_GROUPS) return shape_of(m, groups, LN_BLOCKS);
  Shape s;
  int64_t rows = 16 / groups;
  while (rows > 1 && (m + rows - 1) / rows < 256) rows = (rows + 1) / 2;
  s.rows = (int)rows;
  s.threads = (s.rows * groups * 16 + 63) / 64 * 64;
  s.blocks = (m + s.rows - 1) / s.rows;
  if (s.blocks > LN_BWD_BLOCKS) s.blocks = LN_BWD_BLOCKS;
  return s;
}

// Shares of the rows of k_layernorm_dw: two blocks a compute unit (2048 x 8192, the
// whole pass: 45.0 us, one block 49.4, four 45.3).
int dw_shares(int64_t m, int groups) {
  return (int)std::max<int64_t>(1, std::min<int64_t>((512 + groups - 1) / groups, (m + 15) / 16));
}

template <typename TG, typename TT, typename TD, bool WB>
hipError_t ln_bwd_launch(const LayerNormBwdArgs& a, hipStream_t stream) {
  const Shape s = ln_bwd_shape(a.m, a.groups);
  const size_t lds = (size_t)(s.threads / 16) * (16 * 20 * 4) + 4 * JOIN * sizeof(double);
  const dim3 grid((unsigned)s.blocks), block((unsigned)s.threads);
  if (a.groups <= LN_WIDE_GROUPS) {
    hipLaunchKernelGGL((k_layernorm_bwd<TG, TT, TD, WB, 256, true>), grid, block, lds, stream, a, s.rows, (int64_t)0);
    return hipGetLastError();
  }
  for (int64_t row0 = 0; row0 < a.m; row0 += s.blocks) {
    const dim3 some((unsigned)std::min(s.blocks, a.m - row0));
    hipLaunchKernelGGL((k_layernorm_bwd<TG, TT, TD, WB, 1024, false>), some, block, lds, stream, a, s.rows, row0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename TG, typename TT, typename TD>
hipError_t ln_bwd_weight(const LayerNormBwdArgs& a, hipStream_t stream) {
  return a.gamma.p == nullptr || a.gamma.bf16 ? ln_bwd_launch<TG, TT, TD, true>(a, stream)
                                              : ln_bwd_launch<TG, TT, TD, false>(a, stream);
}

template <typename TG, typename TT>
hipError_t ln_bwd_dx(const LayerNormBwdArgs& a, hipStream_t stream) {
  const hipError_t e =
      a.dx_bf16 ? ln_bwd_weight<TG, TT, uint16_t>(a, stream) : ln_bwd_weight<TG, TT, float>(a, stream);
  if (e != hipSuccess || a.stats == nullptr) return e;
  const int shares = dw_shares(a.m, a.groups);
  hipLaunchKernelGGL((k_layernorm_dw<TG, TT>), dim3((unsigned)(shares * a.groups)), dim3(256), 0, stream, a, shares);
  return hipGetLastError();
}

int64_t partial_rows(int64_t m, int groups) {
  return groups > LN_WIDE_GROUPS ? dw_shares(m, groups) : ln_bwd_shape(m, groups).blocks;
}

}  // namespace

hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t stream) {
  return a.x_bf16 ? ln_x<uint16_t>(a, stream) : ln_x<float>(a, stream);
}

// Partial rows of dgamma and dbeta, then mu and r of each wide row.
int64_t layernorm_bwd_workspace_bytes(int64_t m, int groups) {
  const int64_t part = partial_rows(m, groups) * 2 * groups * 256 * 4;
  return part + (groups > LN_WIDE_GROUPS ? m * 16 : 0);
}

hipError_t launch_layernorm_bwd(const LayerNormBwdArgs& args, hipStream_t stream) {
  LayerNormBwdArgs a = args;
  const int64_t k = (int64_t)a.groups * 256;
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  const int64_t rows = a.m > 0 ? partial_rows(a.m, a.groups) : 0;  // m == 0: none, so the sums are zero
  a.stats = sums && a.groups > LN_WIDE_GROUPS ? (double*)(a.part + rows * 2 * k) : nullptr;
  if (a.m > 0) {
    hipError_t e;
    if (a.dy_bf16)
      e = a.t_bf16 ? ln_bwd_dx<uint16_t, uint16_t>(a, stream) : ln_bwd_dx<uint16_t, float>(a, stream);
    else
      e = a.t_bf16 ? ln_bwd_dx<float, uint16_t>(a, stream) : ln_bwd_dx<float, float>(a, stream);
    if (e != hipSuccess) return e;
  }
  return sums ? launch_colsum(a.part, rows, 2 * k, a.dgamma, k, a.dbeta, stream) : hipSuccess;
}

}  // namespace tp
