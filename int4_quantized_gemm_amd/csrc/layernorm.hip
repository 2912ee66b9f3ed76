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
#include <type_traits>

#include "block_ops.hpp"
#include "e4m3.hpp"
#include "philox.hpp"
#include "row_sets.hpp"

namespace tp {

enum { LN_OUT_I8 = 0, LN_OUT_BF16 = 1, LN_OUT_FP8 = 2 };

// Sum (or maximum) over the threads of a row: all threads of the block call it
// with the same red, which the next join but one may use again.
template <bool MAX>
__device__ __forceinline__ double row_join(double v, const Place& pl, int groups, double* red) {
  v = MAX ? set_max(v) : set_sum(v);
  int first = pl.slot * groups, count = pl.active ? groups : 0;
  if (pl.wide) {  // sets past the row hold zeros
    const double o = swz_xor<16>(v);
    v = MAX ? fmax(v, o) : v + o;
    const double p = __shfl_xor(v, 32);
    v = MAX ? fmax(v, p) : v + p;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    first = 0;
    count = pl.active ? (int)(blockDim.x >> 6) : 0;
  } else if (pl.l16 == 0) {
    red[pl.set] = v;
  }
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < count; ++w) s = MAX ? fmax(s, red[first + w]) : s + red[first + w];
  return s;
}

// ------------------------------------------------------------------ forward
// Codes: fp64 throughout, so they are those of exact arithmetic on the normed
// row. bf16 rows: the deviations and the row factor in fp64, what follows in
// fp32, one rounding.
template <typename TX, typename TS, bool RES, int OUT, int NT>
__global__ __launch_bounds__(NT, 4) void k_layernorm(LayerNormArgs a, int rows_per_block) {
  typedef typename std::conditional<OUT == LN_OUT_BF16, float, double>::type T;
  constexpr int SET_BYTES = 16 * (16 + (sizeof(T) == 4 ? 4 : 2)) * (int)sizeof(T);
  extern __shared__ __align__(16) uint8_t lds[];
  const Place pl = place_of(a.groups, rows_per_block);
  uint8_t* bbuf = lds + pl.set * SET_BYTES;
  T* tbuf = reinterpret_cast<T*>(bbuf);
  const int sets = blockDim.x >> 4;
  double* red = reinterpret_cast<double*>(lds + sets * SET_BYTES);  // [3][sets]
  const int64_t col = (int64_t)pl.grp * 256 + pl.l16 * 8;
  const int64_t k = (int64_t)a.groups * 256;
  const double inv_k = 1.0 / (double)k;
  PhiloxKey key{};
  if (RES && a.drop.rng != nullptr) key = philox_key(a.drop.rng);

  float gm[16], bt[16];
  if (pl.active) {
    load_vec16(a.gamma, col, gm);
    if (a.beta.p != nullptr) load_vec16(a.beta, col, bt);
  }
  if (!pl.active || a.beta.p == nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i) bt[i] = 0.f;
  }
  if (!pl.active) {
#pragma unroll
    for (int i = 0; i < 16; ++i) gm[i] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * pl.rows;
  for (int64_t base = (int64_t)blockIdx.x * pl.rows; base < a.m; base += step) {
    const int64_t row = base + pl.slot;
    const bool live = pl.active && row < a.m;
    Runs<TX> rx;
    Runs<TS> rr;
    if (live) {
      rx.load((const TX*)a.x + row * a.ldx + col);
      if constexpr (RES) rr.load((const TS*)a.res + row * a.ldr + col);
    } else {
      rx.zero();
      if constexpr (RES) rr.zero();
    }
    float t[16];
    if (RES && a.drop.rng != nullptr) {
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

    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += (double)t[i];
    const double mu = row_join<false>(s, pl, a.groups, red) * inv_k;
    s = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const double d = (double)t[i] - mu;
      s = fma(d, d, s);
    }
    if (!pl.active) s = 0.0;
    const double r = 1.0 / sqrt(row_join<false>(s, pl, a.groups, red + sets) * inv_k + a.eps);

    T v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const double n = ((double)t[i] - mu) * r;
      if constexpr (OUT == LN_OUT_BF16)
        v[i] = fmaf((float)n, gm[i], bt[i]);
      else
        v[i] = fma(n, (double)gm[i], (double)bt[i]);
    }
    if (a.rotate) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= (T)0.0625;
      fwht16_regs(v);
      transpose16(v, tbuf, pl.l16);
      fwht16_regs(v);
    }

    if constexpr (OUT == LN_OUT_BF16) {
      if (a.rotate) transpose16_back(v, tbuf, pl.l16);
      if (live) store16((uint16_t*)a.y + row * a.ldy + col, v);
    } else if constexpr (OUT == LN_OUT_FP8) {
      // A set holds two blocks of 128. After the transform its lanes 0 .. 7 hold
      // the first one, register q being element l16 of lane q's two runs;
      // without it the first run of every lane is the first one's.
      uint32_t w[4];
      uint8_t* yrow = (uint8_t*)a.y + row * a.ldy + (int64_t)pl.grp * 256;
      if (a.rotate) {
        double am = absmax16(v);
        am = fmax(am, swz_xor<1>(am));
        am = fmax(am, swz_xor<2>(am));
        am = fmax(am, swz_xor<4>(am));
        const float sc = e4m3_scale(am);
        const double inv = sc > 0.f ? 1.0 / (double)sc : 0.0;
        e4m3_codes<16>(w, [&](int i) { return v[i]; }, [&](int) { return sc; }, [&](int) { return inv; });
        const int at = 128 * (pl.l16 >> 3) + (pl.l16 & 7);
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
          double x[8];
          double am = 0.0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = v[8 * h + j];
            am = absmax2(am, x[j]);
          }
          am = set_max(am);
          const float sc = e4m3_scale(am);
          uint32_t w2[2];
          const double inv = sc > 0.f ? 1.0 / (double)sc : 0.0;
          e4m3_codes<8>(w2, [&](int i) { return x[i]; }, [&](int) { return sc; }, [&](int) { return inv; });
          if (live) {
            *reinterpret_cast<uint2*>(yrow + 128 * h + 8 * pl.l16) = uint2{w2[0], w2[1]};
            if (pl.l16 == 0) a.scales[(2 * pl.grp + h) * a.ldscales + row] = sc;
          }
        }
      }
    } else {
      const double amax = row_join<true>(absmax16(v), pl, a.groups, red + 2 * sets);
      const float s32 = (float)(amax / 127.0);
      const double s64 = (double)s32, inv = s32 > 0.f ? 1.0 / s64 : 0.0;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int q = 0; q < 16; ++q)
        w[q >> 2] |= ((uint32_t)quant_code(v[q], s64, inv, 127.0) & 0xffu) << (8 * (q & 3));
      if (a.rotate) {
        const int at = 128 * (pl.l16 >> 3) + (pl.l16 & 7);
        wave_lds_sync();
#pragma unroll
        for (int q = 0; q < 16; ++q) bbuf[at + 8 * q] = (uint8_t)(w[q >> 2] >> (8 * (q & 3)));
        wave_lds_sync();
        const u32x4_t w4 = *reinterpret_cast<const u32x4_t*>(bbuf + 16 * pl.l16);
        if (live)
          *reinterpret_cast<u32x4_t*>((uint8_t*)a.y + row * a.ldy + (int64_t)pl.grp * 256 + 16 * pl.l16) = w4;
      } else if (live) {
        uint8_t* yp = (uint8_t*)a.y + row * a.ldy + col;
        *reinterpret_cast<uint2*>(yp) = uint2{w[0], w[1]};
        *reinterpret_cast<uint2*>(yp + 128) = uint2{w[2], w[3]};
      }
      if (live && pl.grp == 0 && pl.l16 == 0) a.scales[row] = s32;
    }
  }
}

// ----------------------------------------------------------------- backward
//   g = dy . blockdiag(H / 16) (the rotation is its own inverse), or dy
//   n = (t - mu) r;  w = gamma g
//   dt = r (w - mean(w) - n mean(w n)) + dsum;   dbranch = drop(dt)
//   dgamma = sum over rows of g n;               dbeta = sum over rows of g
// fp32, the row's sums, the deviations and n's product in fp64. A thread keeps
// its 16 columns of dgamma and dbeta over the rows of its block; the blocks'
// sums are joined by k_colsum in a fixed order.
template <typename TG, typename TT, typename TD, int NT>
__global__ __launch_bounds__(NT, 1) void k_layernorm_bwd(LayerNormBwdArgs a, int rows_per_block) {
  constexpr int SET_BYTES = 16 * (16 + 4) * 4;
  extern __shared__ __align__(16) uint8_t lds[];
  const Place pl = place_of(a.groups, rows_per_block);
  float* tbuf = reinterpret_cast<float*>(lds + pl.set * SET_BYTES);
  const int sets = blockDim.x >> 4;
  double* red = reinterpret_cast<double*>(lds + sets * SET_BYTES);  // [4][sets]
  const int64_t col = (int64_t)pl.grp * 256 + pl.l16 * 8;
  const int64_t k = (int64_t)a.groups * 256;
  const double inv_k = 1.0 / (double)k;
  PhiloxKey key{};
  if (a.drop.rng != nullptr) key = philox_key(a.drop.rng);

  float gm[16], dg[16], db[16];
  if (pl.active) {
    load_vec16(a.gamma, col, gm);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) gm[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) dg[i] = db[i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * pl.rows;
  for (int64_t base = (int64_t)blockIdx.x * pl.rows; base < a.m; base += step) {
    const int64_t row = base + pl.slot;
    const bool live = pl.active && row < a.m;
    Runs<TG> rg;
    Runs<TT> rt;
    Runs<TD> rd;
    rd.zero();
    if (live) {
      rg.load((const TG*)a.dy + row * a.lddy + col);
      rt.load((const TT*)a.t + row * a.ldt + col);
      if (a.dsum != nullptr) rd.load((const TD*)a.dsum + row * a.ldds + col);
    } else {
      rg.zero();
      rt.zero();
    }
    double c0 = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) c0 += (double)rt.get(i);
    float g[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = rg.get(i);
    if (a.rotate) {
#pragma unroll
      for (int i = 0; i < 16; ++i) g[i] *= 0.0625f;
      fwht16_regs(g);
      transpose16(g, tbuf, pl.l16);
      fwht16_regs(g);
      transpose16_back(g, tbuf, pl.l16);
    }
    const double mu = row_join<false>(c0, pl, a.groups, red) * inv_k;
    double c1 = 0.0, c2 = 0.0, c3 = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const double d = (double)rt.get(i) - mu, w = (double)(g[i] * gm[i]);
      c1 += w;
      c2 = fma(w, d, c2);
      c3 = fma(d, d, c3);
    }
    if (!pl.active) c3 = 0.0;
    c1 = row_join<false>(c1, pl, a.groups, red + sets);
    c2 = row_join<false>(c2, pl, a.groups, red + 2 * sets);
    c3 = row_join<false>(c3, pl, a.groups, red + 3 * sets);
    const double r64 = 1.0 / sqrt(c3 * inv_k + a.eps);
    const float r = (float)r64, m1 = (float)(c1 * inv_k), m2 = (float)(r64 * (c2 * inv_k));
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float n = (float)(((double)rt.get(i) - mu) * r64);
      o[i] = fmaf(r, fmaf(-n, m2, g[i] * gm[i] - m1), rd.get(i));
      if (live) {
        dg[i] = fmaf(g[i], n, dg[i]);
        db[i] += g[i];
      }
    }
    if (live) {
      store16((TD*)a.dx + row * a.lddx + col, o);
      if (a.dbranch != nullptr) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4_t w = philox4x32_10(key, (uint64_t)(row * k + col + 128 * h) >> 3);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[8 * h + j] = philox_drop(w, j, a.drop, o[8 * h + j]);
        }
        store16((TD*)a.dbranch + row * a.lddb + col, o);
      }
    }
  }
  if (a.dgamma == nullptr && a.dbeta == nullptr) return;
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

// ---------------------------------------------------------------- launchers
namespace {

constexpr int64_t LN_BLOCKS = 65536;    // blocks walk rows beyond that many (threads of a grid in 32 bits)
constexpr int64_t LN_BWD_BLOCKS = 512;  // partial rows of dgamma and dbeta

template <typename TX, typename TS, bool RES, int OUT>
hipError_t ln_launch(const LayerNormArgs& a, hipStream_t stream) {
  const Shape s = shape_of(a.m, a.groups, LN_BLOCKS);
  const int set_bytes = OUT == LN_OUT_BF16 ? 16 * 20 * 4 : 16 * 18 * 8;
  const size_t lds = (size_t)(s.threads / 16) * (set_bytes + 3 * sizeof(double));
  const dim3 grid((unsigned)s.blocks), block((unsigned)s.threads);
  if (s.threads <= 256)
    hipLaunchKernelGGL((k_layernorm<TX, TS, RES, OUT, 256>), grid, block, lds, stream, a, s.rows);
  else
    hipLaunchKernelGGL((k_layernorm<TX, TS, RES, OUT, 1024>), grid, block, lds, stream, a, s.rows);
  return hipGetLastError();
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

Shape ln_bwd_shape(int64_t m, int groups) {
  Shape s;
  int64_t rows = groups <= 16 ? 16 / groups : 1;
  while (rows > 1 && (m + rows - 1) / rows < 256) rows = (rows + 1) / 2;
  s.rows = (int)rows;
  s.threads = (s.rows * groups * 16 + 63) / 64 * 64;
  s.blocks = (m + s.rows - 1) / s.rows;
  if (s.blocks > LN_BWD_BLOCKS) s.blocks = LN_BWD_BLOCKS;
  return s;
}

template <typename TG, typename TT, typename TD>
hipError_t ln_bwd_launch(const LayerNormBwdArgs& a, hipStream_t stream) {
  const Shape s = ln_bwd_shape(a.m, a.groups);
  const size_t lds = (size_t)(s.threads / 16) * (16 * 20 * 4 + 4 * sizeof(double));
  const dim3 grid((unsigned)s.blocks), block((unsigned)s.threads);
  if (s.threads <= 256)
    hipLaunchKernelGGL((k_layernorm_bwd<TG, TT, TD, 256>), grid, block, lds, stream, a, s.rows);
  else
    hipLaunchKernelGGL((k_layernorm_bwd<TG, TT, TD, 1024>), grid, block, lds, stream, a, s.rows);
  return hipGetLastError();
}

template <typename TG, typename TT>
hipError_t ln_bwd_dx(const LayerNormBwdArgs& a, hipStream_t stream) {
  return a.dx_bf16 ? ln_bwd_launch<TG, TT, uint16_t>(a, stream) : ln_bwd_launch<TG, TT, float>(a, stream);
}

}  // namespace

hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t stream) {
  return a.x_bf16 ? ln_x<uint16_t>(a, stream) : ln_x<float>(a, stream);
}

int64_t layernorm_bwd_partial_rows(int64_t m, int groups) { return ln_bwd_shape(m, groups).blocks; }

hipError_t launch_layernorm_bwd(const LayerNormBwdArgs& a, hipStream_t stream) {
  if (a.m > 0) {
    hipError_t e;
    if (a.dy_bf16)
      e = a.t_bf16 ? ln_bwd_dx<uint16_t, uint16_t>(a, stream) : ln_bwd_dx<uint16_t, float>(a, stream);
    else
      e = a.t_bf16 ? ln_bwd_dx<float, uint16_t>(a, stream) : ln_bwd_dx<float, float>(a, stream);
    if (e != hipSuccess) return e;
  }
  if (a.dgamma == nullptr && a.dbeta == nullptr) return hipSuccess;
  // m == 0: no partial rows, so the sums are zero
  const int64_t k = (int64_t)a.groups * 256;
  return launch_colsum(a.part, a.m > 0 ? layernorm_bwd_partial_rows(a.m, a.groups) : 0, 2 * k, a.dgamma, k, a.dbeta,
                       stream);
}

}  // namespace tp
