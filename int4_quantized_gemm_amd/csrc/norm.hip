// Residual addition, RMS norm and rotation of whole rows in front of a
// projection, and their gradients (the TensorFold pull request #948 lists
// RMSNorm and the residual among the row kernels around the projections; the
// residual here is the plain sum, without a gate or modulation).
//
//   t  = stream(x + residual), or x          r = (mean(t^2) + eps)^(-1/2)
//   h  = t r gamma                           h' = h . blockdiag(H / 16)
//
// The row factor r commutes with the rotation, so one pass over the row is
// enough: t gamma is rotated while t^2 is summed, and r multiplies the results.
//
// Work layout: a 256-group is held by a set of 16 lanes, 16 elements each (two
// runs of eight; the butterflies over a lane's registers, a transpose between
// lanes and registers, and the butterflies again are group16.hpp's, whichever
// index bits a lane holds); a row takes one set per group, so a block of up
// to 1024 threads holds a row of up to 64 groups, or several rows of fewer than
// four. Every element is read once; four waves a SIMD hide the loads (a block
// that kept its next row in flight held three waves of 150 registers: 26.6
// against 25.2 us for the codes of 4032 x 3072, 21.3 against 19.4 for rows).
#include <type_traits>

#include "block_ops.hpp"
#include "row_sets.hpp"

namespace tp {

enum { NORM_OUT_I8 = 0, NORM_OUT_BF16 = 1 };

// Whether a lane's set has one of these lanes.
__device__ __forceinline__ bool reaches(uint64_t lanes, int lane) { return ((lanes >> (lane & 48)) & 0xffff) != 0; }

// ------------------------------------------------------------------ forward
// int8: the transform, the row maximum and the codes in fp64, as the library's
// quantizer does (its codes are those of exact arithmetic on the normed row:
// t gamma is exact in fp64, nothing is rounded to a shorter type in between).
// bf16: fp32 arithmetic, one rounding.
//
// Bound by HBM for the bf16 rows (4096 x 3072, bf16 in and stream: 18.8 us, 5.3
// TB/s) and by fp64 issue plus the row's chain (load, transpose, two joins, two
// divisions) for the codes (4032 x 3072, fp32 in, bf16 stream: 24.7 us, 4.5 TB/s;
// 4096 x 8192 58.6 us, 5.1 TB/s; 1024 x 12288, whose 112 KiB of LDS leave one block a
// compute unit, 31.8 us, 3.6 TB/s).
template <typename TX, typename TS, bool RES, int OUT, int NT>
__global__ __launch_bounds__(NT, 4) void k_norm_rotate(NormArgs a, int rows_per_block) {
  typedef typename std::conditional<OUT == NORM_OUT_I8, double, float>::type T;
  constexpr int SET_BYTES = 16 * (16 + (sizeof(T) == 4 ? 4 : 2)) * (int)sizeof(T);
  extern __shared__ __align__(16) uint8_t lds[];
  const Place pl = place_of(a.groups, rows_per_block);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint8_t* bbuf = lds + pl.set * SET_BYTES;
  T* tbuf = reinterpret_cast<T*>(bbuf);
  double2* red = reinterpret_cast<double2*>(lds + (blockDim.x >> 4) * SET_BYTES);  // [2][sets]
  const int sets = blockDim.x >> 4, waves = blockDim.x >> 6;
  const int64_t col = (int64_t)pl.grp * 256 + pl.l16 * 8;
  const double inv_k = 1.0 / (double)(a.groups * 256);
  const double unscale = a.rotate ? 0.0625 : 1.0;

  float gm[16];
  if (pl.active) {
    load_vec16(a.gamma, col, gm);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) gm[i] = 0.f;
  }
  Runs<TX> rx;
  Runs<TS> rr;
  auto fetch = [&](int64_t row) {
    if (pl.active && row < a.m) {
      rx.load((const TX*)a.x + row * a.ldx + col);
      if constexpr (RES) rr.load((const TS*)a.res + row * a.ldr + col);
    } else {
      rx.zero();
      if constexpr (RES) rr.zero();
    }
  };
  const int64_t step = (int64_t)gridDim.x * pl.rows;
  int parity = 0;
  for (int64_t base = (int64_t)blockIdx.x * pl.rows; base < a.m; base += step, parity ^= 1) {
    const int64_t row = base + pl.slot;
    const bool live = pl.active && row < a.m;
    fetch(row);
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = RES ? as_stream<TS>(rx.get(i) + rr.get(i)) : rx.get(i);
    if (RES && live) store16((TS*)a.sum + row * a.ldsum + col, t);

    T v[16];
    double ss = 0.0, amax = 0.0;
    uint64_t over = 0;  // lanes with a value past 2^116 (bf16 rows)
    if constexpr (OUT == NORM_OUT_I8) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double td = (double)t[i];
        asm volatile("" : "+v"(gm[i]));  // widened here, not kept as 32 registers of fp64
        ss = fma(td, td, ss);
        v[i] = td * (double)gm[i];
      }
      asm volatile("" : "+v"(ss));  // summed here, not with t kept through the transform
    } else {
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double td = (double)t[i];  // squares up to 2^256: no overflow
        ss = fma(td, td, ss);
        v[i] = t[i] * gm[i];
        most = fmaxf(most, fabsf(v[i]));
      }
      // Sums of 256 values of up to 2^128 leave fp32: a group that reaches 2^116
      // goes through the transform as 2^-12 of itself. That is exact: what falls
      // below fp32's steps there is below bf16's after the row factor. (The test
      // costs 4096 x 3072 rows up to 0.2 of 12.5 to 35 us, 1024 x 12288 0.3 of 26.6.)
      over = __ballot(most >= 0x1p116f);
      asm volatile("" : "+v"(ss));  // summed here
      if (over != 0) {
        const float sink = reaches(over, lane) ? 0x1p-12f : 1.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= sink;
      }
    }
    if (a.rotate) {
      fwht16_regs(v);
      transpose16(v, tbuf, pl.l16);
      fwht16_regs(v);
    } else if (OUT == NORM_OUT_I8) {
      transpose16(v, tbuf, pl.l16);  // the same output order either way
    }
    if constexpr (OUT == NORM_OUT_I8) amax = set_max(absmax16(v));
    ss = set_sum(ss);
    double2* rp = red + parity * sets;
    int first = pl.slot * a.groups, count = a.groups;
    if (pl.wide) {  // sets past the row hold zeros
      ss += swz_xor<16>(ss);
      ss += __shfl_xor(ss, 32);
      if constexpr (OUT == NORM_OUT_I8) {
        amax = fmax(amax, swz_xor<16>(amax));
        amax = fmax(amax, __shfl_xor(amax, 32));
      }
      if (lane == 0) rp[wave] = double2{ss, amax};
      first = 0;
      count = waves;
    } else if (pl.l16 == 0) {
      rp[pl.set] = double2{ss, amax};
    }
    __syncthreads();  // (the other parity's entries may still be read by slower waves)
    if (!pl.active) {
      first = 0;
      count = 0;
    }
    ss = 0.0;
    amax = 0.0;
    for (int w = 0; w < count; ++w) {
      const double2 e = rp[first + w];
      ss += e.x;
      amax = fmax(amax, e.y);
    }
    const double r = 1.0 / sqrt(ss * inv_k + a.eps);

    if constexpr (OUT == NORM_OUT_I8) {
      const double unit = r * unscale;  // the values above times this are the rotated, normed row
      const float s = (float)(amax * unit / 127.0);
      const double s64 = (double)s;
      const double inv64 = s > 0.0f ? 1.0 / s64 : 0.0;
      const double invu = inv64 * unit;
      constexpr double MAGIC = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer (RNE)
      // As in k_rotq_i8_d: the product with invu decides the code unless it is
      // within 1e-9 of a tie; rows with a subnormal scale take the division.
      const bool direct = s == 0.0f || s >= 0x1p-126f;
      // after the transpose register q is element l16 of lane q's two runs
      const int at = 128 * (pl.l16 >> 3) + (pl.l16 & 7);
      wave_lds_sync();
      bool tie = false;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const double f = fma(v[q], invu, MAGIC);
        const double d = fma(v[q], invu, MAGIC - f);
        tie |= !(fabs(d) < 0.5 - 1e-9);
        bbuf[at + 8 * q] = (uint8_t)__builtin_bit_cast(uint64_t, f);
        if ((q & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // four codes at a time: fewer registers
      }
      if (__ballot((tie || !direct) && live)) {
        double invr = invu;
        asm volatile("" : "+v"(invr));  // recomputed: the first pass's values need not stay in registers
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const double f = fma(v[q], invr, MAGIC);
          const double d = fma(v[q], invr, MAGIC - f);
          if (!direct || !(fabs(d) < 0.5 - 1e-9))
            bbuf[at + 8 * q] = (uint8_t)quant_code(v[q] * unit, s64, inv64, 127.0);
          __builtin_amdgcn_sched_barrier(0);  // one division at a time
        }
      }
      wave_lds_sync();
      const u32x4_t w4 = *reinterpret_cast<const u32x4_t*>(bbuf + 16 * pl.l16);
      if (live) {
        *reinterpret_cast<u32x4_t*>((int8_t*)a.y + row * a.ldy + (int64_t)pl.grp * 256 + 16 * pl.l16) = w4;
        if (pl.grp == 0 && pl.l16 == 0) a.scales[row] = s;
      }
    } else {
      const float unit = (float)(r * (over != 0 && reaches(over, lane) ? 4096.0 * unscale : unscale));
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= unit;
      if (a.rotate) transpose16_back(v, tbuf, pl.l16);
      if (live) store16((uint16_t*)a.y + row * a.ldy + col, v);
    }
  }
}

// ----------------------------------------------------------------- backward
//   g = dy . blockdiag(H / 16) (the rotation is its own inverse), or dy
//   n = t r;   dt = r (gamma g - n r mean(gamma g t)) + dsum;   dgamma = sum over rows of g n
// in fp32, the two sums of a row in fp64: n, r mean(.) and the difference are of
// the gradients' size for rows of any size (t r^3 mean(.) taken as such leaves
// fp32 from rows of 1e21 on). A thread keeps its 16 columns of dgamma over the rows of its block;
// the blocks' sums are joined by k_colsum in a fixed order. Bound by HBM (4096 x
// 3072, fp32 dy, bf16 t, dsum and dx: 25.7 us, 4.9 TB/s, and 4.7 us for the join
// of 512 partial rows). Rows of more than 16 groups with a block each (ONE) keep
// no sums, so that two of 768 threads share a compute unit; their partial rows,
// one a row, are written and read besides (333 x 12288 fp32: 15.7 us and 4.4 for
// the join). A stream gradient does not fit there: those forms spill 4 to 14 of
// their 80 registers (the same with it 21.8 and 4.4 us, 3.0 TB/s), and the ones
// of several wide rows a block 2 to 8 of 128 (bf16 with it, 4096 x 5120: 36.4 us,
// 4.6 TB/s; 4096 x 8192: 49.8 us, 5.4 TB/s; 1000 x 12288 with an fp32 dy: 34.1 us,
// 3.6 TB/s).
template <typename TG, typename TT, typename TD, bool DS, int NT, bool ONE>
__global__ __launch_bounds__(NT, NT == 768 ? 6 : 1) void k_norm_bwd(NormBwdArgs a, int rows_per_block) {
  constexpr int SET_BYTES = 16 * (16 + 4) * 4;
  extern __shared__ __align__(16) uint8_t lds[];
  const Place pl = place_of(a.groups, rows_per_block);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* tbuf = reinterpret_cast<float*>(lds + pl.set * SET_BYTES);
  double2* red = reinterpret_cast<double2*>(lds + (blockDim.x >> 4) * SET_BYTES);  // [2][sets]
  const int sets = blockDim.x >> 4, waves = blockDim.x >> 6;
  const int64_t col = (int64_t)pl.grp * 256 + pl.l16 * 8;
  const double inv_k = 1.0 / (double)(a.groups * 256);

  float gm[16], dg[16];
  if (pl.active) {
    load_vec16(a.gamma, col, gm);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) gm[i] = 0.f;
  }
  if constexpr (!ONE) {
#pragma unroll
    for (int i = 0; i < 16; ++i) dg[i] = 0.f;
  }
  Runs<TG> rg;
  Runs<TT> rt;
  Runs<TD> rd;
  auto fetch = [&](int64_t row) {
    if (pl.active && row < a.m) {
      rg.load((const TG*)a.dy + row * a.lddy + col);
      rt.load((const TT*)a.t + row * a.ldt + col);
      if constexpr (DS) rd.load((const TD*)a.dsum + row * a.ldds + col);
    } else {
      rg.zero();
      rt.zero();
      if constexpr (DS) rd.zero();
    }
  };
  const int64_t step = (int64_t)gridDim.x * pl.rows;
  int parity = 0;
  // Rows of more than 16 groups leave a thread 128 registers: no row is kept
  // in flight there.
  constexpr bool AHEAD = NT <= 256 && !ONE;
  if (AHEAD) fetch((int64_t)blockIdx.x * pl.rows + pl.slot);
  for (int64_t base = (int64_t)blockIdx.x * pl.rows; base < a.m; base += step, parity ^= 1) {
    const int64_t row = base + pl.slot;
    const bool live = pl.active && row < a.m;
    if (!AHEAD) fetch(row);
    float g[16], t[16], d[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      g[i] = rg.get(i);
      t[i] = rt.get(i);
      d[i] = DS ? rd.get(i) : 0.f;
    }
    if (AHEAD && base + step < a.m) fetch(row + step);
    if (a.rotate) {
      fwht16_regs(g);
      transpose16(g, tbuf, pl.l16);
      fwht16_regs(g);
      transpose16_back(g, tbuf, pl.l16);
#pragma unroll
      for (int i = 0; i < 16; ++i) g[i] *= 0.0625f;
    }
    double c1 = 0.0, c2 = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const double td = (double)t[i];
      c1 = fma((double)(g[i] * gm[i]), td, c1);  // up to 2^256, as the squares
      c2 = fma(td, td, c2);
    }
    asm volatile("" : "+v"(c1), "+v"(c2));  // summed here
    c1 = set_sum(c1);
    c2 = set_sum(c2);
    double2* rp = red + parity * sets;
    int first = pl.slot * a.groups, count = a.groups;
    if (pl.wide) {
      c1 += swz_xor<16>(c1);
      c1 += __shfl_xor(c1, 32);
      c2 += swz_xor<16>(c2);
      c2 += __shfl_xor(c2, 32);
      if (lane == 0) rp[wave] = double2{c1, c2};
      first = 0;
      count = waves;
    } else if (pl.l16 == 0) {
      rp[pl.set] = double2{c1, c2};
    }
    __syncthreads();
    if (!pl.active) {
      first = 0;
      count = 0;
    }
    double s1 = 0.0, s2 = 0.0;
    for (int w = 0; w < count; ++w) {
      const double2 e = rp[first + w];
      s1 += e.x;
      s2 += e.y;
    }
    const double rd64 = 1.0 / sqrt(s2 * inv_k + a.eps);
    const float r = (float)rd64;
    const float mean = (float)(rd64 * (s1 * inv_k));
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float n = t[i] * r;
      o[i] = fmaf(r, fmaf(-n, mean, g[i] * gm[i]), d[i]);
      dg[i] = ONE ? g[i] * n : fmaf(g[i], n, dg[i]);
    }
    if (live) store16((TD*)a.dx + row * a.lddx + col, o);
    if (ONE) break;
  }
  if (a.dgamma == nullptr) return;
  float* part = a.part + (int64_t)blockIdx.x * (a.groups * 256);
  if (pl.rows == 1) {
    if (pl.active) store16(part + col, dg);
    return;
  }
  // the sums of the block's rows, added in order
  float* sums = reinterpret_cast<float*>(lds);  // [rows][columns]: 1 KiB of a set's 1.25 KiB
  __syncthreads();
  if (pl.active) store16(sums + pl.slot * (a.groups * 256) + col, dg);
  __syncthreads();
  for (int c = threadIdx.x; c < a.groups * 256; c += (int)blockDim.x) {
    float s = sums[c];
    for (int w = 1; w < pl.rows; ++w) s += sums[w * (a.groups * 256) + c];
    part[c] = s;
  }
}

// Column sums of part [rows, cols]: 64 columns a block, 16 slices of the rows,
// the slices joined in order. The first columns go to out, the others to out2
// (either may be null).
__global__ __launch_bounds__(1024) void k_colsum(const float* __restrict__ part, int64_t rows, int64_t cols,
                                                 float* __restrict__ out, int64_t first, float* __restrict__ out2) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, sl = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + c;
  const int64_t r0 = rows * sl / 16, r1 = rows * (sl + 1) / 16;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 16
    for (int64_t r = r0; r < r1; ++r) s += part[r * cols + col];
  }
  red[sl][c] = s;
  __syncthreads();
  if (sl == 0 && col < cols) {
    s = red[0][c];
#pragma unroll
    for (int w = 1; w < 16; ++w) s += red[w][c];
    if (col < first) {
      if (out != nullptr) out[col] = s;
    } else if (out2 != nullptr) {
      out2[col - first] = s;
    }
  }
}

// ---------------------------------------------------------------- launchers
namespace {

constexpr int64_t NORM_BLOCKS = 65536;  // blocks walk rows beyond that many (threads of a grid in 32 bits)
// More blocks hide more of a row's chain, fewer write fewer partial rows of dgamma.
// bf16 with dsum, the join included: 4096 x 3072 28.4 us, 36.2 with 256 blocks, 30.3
// with 1024; 12288 x 1024 27.7, 30.1, 32.2; 1024 x 3072 13.5, 14.2, 15.4. Wide rows
// alone would do with 256 (1000 x 12288, fp32 dy: 40.8, 35.8, 49.6).
constexpr int64_t NORM_BWD_BLOCKS = 512;

template <typename TX, typename TS, bool RES, int OUT>
hipError_t norm_launch(const NormArgs& a, hipStream_t stream) {
  const Shape s = shape_of(a.m, a.groups, NORM_BLOCKS);
  const int set_bytes = OUT == NORM_OUT_I8 ? 16 * 18 * 8 : 16 * 20 * 4;
  const size_t lds = (size_t)(s.threads / 16) * (set_bytes + 2 * sizeof(double2));
  const dim3 grid((unsigned)s.blocks), block((unsigned)s.threads);
  if (s.threads <= 256)
    hipLaunchKernelGGL((k_norm_rotate<TX, TS, RES, OUT, 256>), grid, block, lds, stream, a, s.rows);
  else
    hipLaunchKernelGGL((k_norm_rotate<TX, TS, RES, OUT, 1024>), grid, block, lds, stream, a, s.rows);
  return hipGetLastError();
}

template <typename TX, typename TS, bool RES>
hipError_t norm_out(const NormArgs& a, hipStream_t stream) {
  return a.out_i8 ? norm_launch<TX, TS, RES, NORM_OUT_I8>(a, stream) : norm_launch<TX, TS, RES, NORM_OUT_BF16>(a, stream);
}

template <typename TX>
hipError_t norm_x(const NormArgs& a, hipStream_t stream) {
  if (a.res == nullptr) return norm_out<TX, float, false>(a, stream);
  return a.s_bf16 ? norm_out<TX, uint16_t, true>(a, stream) : norm_out<TX, float, true>(a, stream);
}

// Short rows share blocks of 16 sets: dgamma's partial sums are one row a block
// however many rows share it, and blocks of one short row leave compute units
// idle. 49152 x 256 bf16: 24.6 us with dgamma's join, 44.5 with blocks of 64
// threads and a partial row each; 12288 x 1024: 23.4 and 42.7. Few rows are spread
// over at least 256 blocks, one a compute unit (256 x 1024: 6.5 us, 8.4 over 128;
// 1024 x 1024: 8.4, 9.8 over 512).
Shape bwd_shape_of(int64_t m, int groups) {
  Shape s;
  int64_t rows = groups <= 16 ? 16 / groups : 1;
  while (rows > 1 && (m + rows - 1) / rows < 256) rows = (rows + 1) / 2;
  s.rows = (int)rows;
  s.threads = (s.rows * groups * 16 + 63) / 64 * 64;
  s.blocks = (m + s.rows - 1) / s.rows;
  if (s.blocks > NORM_BWD_BLOCKS) s.blocks = NORM_BWD_BLOCKS;
  return s;
}

template <typename TG, typename TT, typename TD, bool DS>
hipError_t bwd_launch(const NormBwdArgs& a, hipStream_t stream) {
  const Shape s = bwd_shape_of(a.m, a.groups);
  const bool one = s.blocks * s.rows >= a.m;
  const size_t lds = (size_t)(s.threads / 16) * (16 * 20 * 4 + 2 * sizeof(double2));
  const dim3 grid((unsigned)s.blocks), block((unsigned)s.threads);
  if (s.threads <= 256)
    hipLaunchKernelGGL((k_norm_bwd<TG, TT, TD, DS, 256, false>), grid, block, lds, stream, a, s.rows);
  else if (one && s.threads <= 768)
    hipLaunchKernelGGL((k_norm_bwd<TG, TT, TD, DS, 768, true>), grid, block, lds, stream, a, s.rows);
  else
    hipLaunchKernelGGL((k_norm_bwd<TG, TT, TD, DS, 1024, false>), grid, block, lds, stream, a, s.rows);
  return hipGetLastError();
}

template <typename TG, typename TT>
hipError_t bwd_dx(const NormBwdArgs& a, hipStream_t stream) {
  if (a.dsum != nullptr)
    return a.dx_bf16 ? bwd_launch<TG, TT, uint16_t, true>(a, stream) : bwd_launch<TG, TT, float, true>(a, stream);
  return a.dx_bf16 ? bwd_launch<TG, TT, uint16_t, false>(a, stream) : bwd_launch<TG, TT, float, false>(a, stream);
}

}  // namespace

hipError_t launch_norm_rotate(const NormArgs& a, hipStream_t stream) {
  return a.x_bf16 ? norm_x<uint16_t>(a, stream) : norm_x<float>(a, stream);
}

int64_t norm_bwd_partial_rows(int64_t m, int groups) { return bwd_shape_of(m, groups).blocks; }

hipError_t launch_colsum(const float* part, int64_t rows, int64_t cols, float* out, int64_t first, float* out2,
                         hipStream_t stream) {
  hipLaunchKernelGGL(k_colsum, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, stream, part, rows, cols, out,
                     first, out2);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t stream) {
  if (a.m > 0) {
    hipError_t e;
    if (a.dy_bf16)
      e = a.t_bf16 ? bwd_dx<uint16_t, uint16_t>(a, stream) : bwd_dx<uint16_t, float>(a, stream);
    else
      e = a.t_bf16 ? bwd_dx<float, uint16_t>(a, stream) : bwd_dx<float, float>(a, stream);
    if (e != hipSuccess) return e;
  }
  if (a.dgamma == nullptr) return hipSuccess;
  // m == 0: no partial rows, so the sum is zero
  const int64_t k = (int64_t)a.groups * 256;
  return launch_colsum(a.part, a.m > 0 ? norm_bwd_partial_rows(a.m, a.groups) : 0, k, a.dgamma, k, nullptr, stream);
}

}  // namespace tp
