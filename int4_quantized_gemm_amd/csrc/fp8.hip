// Quantizers of the 8-bit float product (fp8_gemm.hip): e4m3 codes with a scale
// per 128 elements of a row, per 128 elements of a column (the codes then lie
// transposed, for a product that sums over the rows), or per 128 x 128 block
// (weights; as they are and transposed).
//
//   s = fp32(amax / 448)    code = e4m3(x / s), nearest even, saturated
//
// computed in fp64, so codes and scales are those of exact arithmetic on x (or
// on its rotation).
//
// A block of 512 threads takes a tile of 128 rows and 256 columns: 32 sets of
// 16 lanes (row_sets.hpp), four consecutive rows each, so that a lane holds the
// codes of four rows of a column as one dword when it turns the tile through
// LDS. Row codes are written as the tile is read; column and block maxima are
// taken on that first pass and their codes on a second one, which finds the
// tile in L2.
#include "block_ops.hpp"
#include "e4m3.hpp"
#include "row_sets.hpp"

namespace tp {

namespace {

constexpr int Q_SETS = 32, Q_ROWS = 128, Q_COLS = 256;
constexpr int Q_PITCH = 33;  // dwords of a column's 128 codes in LDS

// Element i of a lane: its column in the tile, after the transform or without.
template <bool ROT>
__device__ __forceinline__ int col_of(int l16, int i) {
  return ROT ? 128 * (l16 >> 3) + (l16 & 7) + 8 * i : 128 * (i >> 3) + 8 * l16 + (i & 7);
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

// The lane's two runs of a row, zeros past the row's end.
template <typename TX>
__device__ __forceinline__ void load_tail(const TX* p, int64_t left, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (128 * h + 8 <= left) {
      float u[8];
      load8(p + 128 * h, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * h + j] = u[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * h + j] = 128 * h + j < left ? widen(p[128 * h + j]) : 0.f;
    }
  }
}

}  // namespace

template <typename TX, bool ROT>
__global__ __launch_bounds__(512) void k_quant_fp8(QuantFp8Args a, int64_t tiles_k, int rows_per_block) {
  constexpr int SET_BYTES = 16 * 18 * 8;
  __shared__ __align__(16) uint8_t turn[ROT ? Q_SETS * SET_BYTES : 16];
  __shared__ double part[8][Q_COLS];
  __shared__ float scale[Q_COLS];
  __shared__ double inverse[Q_COLS];
  __shared__ uint32_t cols[Q_COLS * Q_PITCH];
  const int l16 = threadIdx.x & 15, set = threadIdx.x >> 4, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t tile_m = blockIdx.x / tiles_k, tile_k = blockIdx.x - tile_m * tiles_k;
  const int64_t r0 = tile_m * rows_per_block, c0 = tile_k * Q_COLS;
  const int64_t kp = (a.k + 127) / 128 * 128;
  const int per_set = rows_per_block / Q_SETS;
  uint8_t* bbuf = turn + (ROT ? set * SET_BYTES : 0);
  double v[16];

  auto fetch = [&](int64_t row) {
    float f[16];
    if (row < a.m) {
      load_tail((const TX*)a.x + row * a.ldx + c0 + 8 * l16, a.k - c0 - 8 * l16, f);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = (double)f[i];
    if constexpr (ROT) {
      fwht16_regs(v);
      transpose16(v, reinterpret_cast<double*>(bbuf), l16);
      fwht16_regs(v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= 0.0625;
    }
  };
  // The codes of a row as they lie in memory.
  auto store_row = [&](int64_t row, const uint32_t (&w)[4]) {
    uint8_t* q = a.q + row * a.ldq + c0;
    if constexpr (ROT) {
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < 16; ++i) bbuf[col_of<true>(l16, i)] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
      wave_lds_sync();
      const u32x4_t w4 = *reinterpret_cast<const u32x4_t*>(bbuf + 16 * l16);
      if (row < a.m) *reinterpret_cast<u32x4_t*>(q + 16 * l16) = w4;
    } else if (row < a.m) {
      if (c0 < kp) *reinterpret_cast<uint2*>(q + 8 * l16) = uint2{w[0], w[1]};
      if (c0 + 128 < kp) *reinterpret_cast<uint2*>(q + 128 + 8 * l16) = uint2{w[2], w[3]};
    }
  };

  const bool by_row = !a.blocks && a.q != nullptr, by_col = !a.blocks && a.qt != nullptr;
  double cm[16], bm[2] = {0.0, 0.0};
#pragma unroll
  for (int i = 0; i < 16; ++i) cm[i] = 0.0;
#pragma unroll 1
  for (int it = 0; it < per_set; ++it) {
    const int64_t row = r0 + set * per_set + it;
    fetch(row);
    if (by_col) {
#pragma unroll
      for (int i = 0; i < 16; ++i) cm[i] = absmax2(cm[i], v[i]);
    }
    if (by_row || a.blocks) {
      double am[2];
      if constexpr (ROT) {  // lanes 0 .. 7 hold the first 128 columns
        am[0] = absmax16(v);
        am[0] = fmax(am[0], swz_xor<1>(am[0]));
        am[0] = fmax(am[0], swz_xor<2>(am[0]));
        am[0] = fmax(am[0], swz_xor<4>(am[0]));
        am[1] = am[0];
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          am[h] = 0.0;
#pragma unroll
          for (int j = 0; j < 8; ++j) am[h] = absmax2(am[h], v[8 * h + j]);
          am[h] = set_max(am[h]);
        }
      }
      bm[0] = fmax(bm[0], am[0]);
      bm[1] = fmax(bm[1], am[1]);
      if (by_row) {
        const float s[2] = {e4m3_scale(am[0]), e4m3_scale(am[1])};
        const double inv[2] = {s[0] > 0.f ? 1.0 / (double)s[0] : 0.0, s[1] > 0.f ? 1.0 / (double)s[1] : 0.0};
        uint32_t w[4];
        e4m3_codes<16>(w, [&](int i) { return v[i]; }, [&](int i) { return s[i >> 3]; },
                       [&](int i) { return inv[i >> 3]; });
        store_row(row, w);
        const int h = ROT ? l16 >> 3 : l16 & 1;
        if (row < a.m && l16 == (ROT ? 8 * h : h) && c0 + 128 * h < kp)
          a.s[(c0 / 128 + h) * a.lds + row] = ROT ? s[0] : (h ? s[1] : s[0]);
      }
    }
  }
  if (!a.blocks && !by_col) return;

  // the tile's scales
  if (a.blocks) {
    if constexpr (ROT) {
      const double o = swz_xor<8>(bm[0]);
      bm[1] = (l16 & 8) ? bm[0] : o;
      bm[0] = (l16 & 8) ? o : bm[0];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bm[h] = fmax(bm[h], swz_xor<16>(bm[h]));
      bm[h] = fmax(bm[h], __shfl_xor(bm[h], 32));
      if (lane == 0) part[wave][h] = bm[h];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      cm[i] = fmax(cm[i], swz_xor<16>(cm[i]));
      cm[i] = fmax(cm[i], __shfl_xor(cm[i], 32));
      if (lane < 16) part[wave][col_of<ROT>(l16, i)] = cm[i];
    }
  }
  __syncthreads();
  if (threadIdx.x < Q_COLS) {
    const int at = a.blocks ? threadIdx.x >> 7 : threadIdx.x;
    double m = part[0][at];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = fmax(m, part[w][at]);
    const float s = e4m3_scale(m);
    scale[threadIdx.x] = s;
    inverse[threadIdx.x] = s > 0.f ? 1.0 / (double)s : 0.0;
    const int64_t col = c0 + threadIdx.x;
    if (a.blocks) {
      if ((threadIdx.x & 127) == 0 && col < kp) {
        if (a.q != nullptr) a.s[tile_m * a.lds + col / 128] = s;
        if (a.qt != nullptr) a.st[col / 128 * a.ldst + tile_m] = s;
      }
    } else if (col < a.k) {
      a.st[tile_m * a.ldst + col] = s;
    }
  }
  __syncthreads();

  uint32_t pack[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) pack[i] = 0u;
#pragma unroll 1
  for (int it = 0; it < per_set; ++it) {
    const int64_t row = r0 + set * per_set + it;
    fetch(row);
    uint32_t w[4];
    e4m3_codes<16>(w, [&](int i) { return v[i]; }, [&](int i) { return scale[col_of<ROT>(l16, i)]; },
                   [&](int i) { return inverse[col_of<ROT>(l16, i)]; });
    if (a.blocks && a.q != nullptr) store_row(row, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) pack[i] |= ((w[i >> 2] >> (8 * (i & 3))) & 0xffu) << (8 * it);
  }
  if (a.qt == nullptr) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) cols[col_of<ROT>(l16, i) * Q_PITCH + set] = pack[i];
  __syncthreads();
  // eight lanes a column, 16 codes each
  for (int c = threadIdx.x >> 3; c < Q_COLS; c += 64) {
    const int64_t col = c0 + c;
    const uint32_t* p = cols + c * Q_PITCH + 4 * (threadIdx.x & 7);
    const u32x4_t w = {p[0], p[1], p[2], p[3]};
    if (col < a.k) *reinterpret_cast<u32x4_t*>(a.qt + col * a.ldqt + r0 + 16 * (threadIdx.x & 7)) = w;
  }
}

namespace {

template <typename TX>
hipError_t quant_launch(const QuantFp8Args& a, hipStream_t stream) {
  // rows alone need no tile of 128 of them: a row a set
  const int rows = a.blocks || a.qt != nullptr ? Q_ROWS : Q_SETS;
  const int64_t tiles_k = (a.k + Q_COLS - 1) / Q_COLS, tiles_m = (a.m + rows - 1) / rows;
  const dim3 grid((unsigned)(tiles_m * tiles_k));
  if (a.rotate)
    hipLaunchKernelGGL((k_quant_fp8<TX, true>), grid, dim3(512), 0, stream, a, tiles_k, rows);
  else
    hipLaunchKernelGGL((k_quant_fp8<TX, false>), grid, dim3(512), 0, stream, a, tiles_k, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(const QuantFp8Args& a, hipStream_t stream) {
  return a.x_bf16 ? quant_launch<uint16_t>(a, stream) : quant_launch<float>(a, stream);
}

}  // namespace tp
