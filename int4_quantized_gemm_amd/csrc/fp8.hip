// Quantizers of the 8-bit float product (fp8_gemm.hip): e4m3 codes with a scale
// per 128 elements of a row, per 128 elements of a column (the codes then lie
// transposed, for a product that sums over the rows), or per 128 x 128 block
// (weights; as they are and transposed).
//
//   s = fp32(amax / 448)    code = e4m3(x / s), nearest even, saturated
//
// Codes and scales are those of exact arithmetic on x (e4m3.hpp), or on its
// rotation in fp64. Everything is read once: what a tile's scales are taken
// from stays in registers until its codes are made.
#include "block_ops.hpp"
#include "e4m3.hpp"
#include "lanes.hpp"
#include "row_sets.hpp"

namespace tp {

namespace {

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

// Eight elements of a row, zeros from the left-th on.
template <typename TX>
__device__ __forceinline__ void load_left(const TX* p, int64_t left, float (&v)[8]) {
  if (left >= 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < left ? widen(p[j]) : 0.f;
  }
}

__device__ __forceinline__ float max8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  return m;
}

// What the codes need of a column's scale, made once for a tile.
struct Inverses {
  float s[256], lo[256], hi[256];
  __device__ __forceinline__ void put(int c, const E4m3Inverse& v) {
    s[c] = v.s;
    lo[c] = v.lo;
    hi[c] = v.hi;
  }
  __device__ __forceinline__ E4m3Inverse get(int c) const { return E4m3Inverse{s[c], lo[c], hi[c]}; }
};

// The codes of eight values of one block.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const E4m3Inverse& s) {
  uint32_t w[2];
  e4m3_codes<8>(w, [&](int i) { return v[i]; }, [&](int i) { return (double)v[i]; }, [&](int) { return s; },
                s.slow());
  return uint2{w[0], w[1]};
}

// Four rows of four codes each as four columns.
__device__ __forceinline__ void turn4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&t)[4]) {
  const uint32_t p = __builtin_amdgcn_perm(b, a, 0x05010400u), q = __builtin_amdgcn_perm(d, c, 0x05010400u);
  const uint32_t r = __builtin_amdgcn_perm(b, a, 0x07030602u), s = __builtin_amdgcn_perm(d, c, 0x07030602u);
  t[0] = __builtin_amdgcn_perm(q, p, 0x05040100u);
  t[1] = __builtin_amdgcn_perm(q, p, 0x07060302u);
  t[2] = __builtin_amdgcn_perm(s, r, 0x05040100u);
  t[3] = __builtin_amdgcn_perm(s, r, 0x07060302u);
}

constexpr int Q_ROWS = 128;  // rows of a tile whose columns or blocks are quantized
constexpr int Q_PITCH = 33;  // dwords of a column's 128 codes in LDS

}  // namespace

// Row codes: a set of 16 lanes takes 128 columns of a row, a block 16 rows. 4096 x
// 4096 bf16 14.1 us (50 MB, 3.6 TB/s; the vector unit is busy 65% of the time, two
// waves in three take the division of some value), fp32 13.3 us (6.3 TB/s; busy 35%,
// as few divisions as e4m3.hpp says). Two or four rows of a set in
// flight: 15.3 and 17.6 us, 2000 x 4096 9.9 and 10.6 against 8.9; ahead only from
// some 10^8 elements on (16384 x 12288 136 and 134 against 144).
template <typename TX>
__global__ __launch_bounds__(256) void k_fp8_rows(QuantFp8Args a, uint32_t blocks_k) {
  const int l16 = threadIdx.x & 15;
  const uint32_t tile = blockIdx.x / blocks_k, g = blockIdx.x - tile * blocks_k;
  const int64_t row = (int64_t)tile * 16 + (threadIdx.x >> 4), col = (int64_t)g * 128 + 8 * l16;
  if (row >= a.m) return;
  float v[8];
  load_left((const TX*)a.x + row * a.ldx + col, a.k - col, v);
  const float s = e4m3_scale(row_all<true>(max8(v)));
  *reinterpret_cast<uint2*>(a.q + row * a.ldq + col) = codes8(v, e4m3_inverse(s));
  if (l16 == 0) a.s[g * a.lds + row] = s;
}

// A tile of 128 rows and 128 columns: 32 sets of 16 lanes, four consecutive rows
// each, so that a lane holds the codes of four rows of a column as one dword
// when it turns the tile through LDS. Bound by its phases (load, maxima, barrier,
// inverses, barrier, codes, turn, barrier, store), which little else covers: two
// blocks a compute unit, the waves wait for 50 to 60% of their time, the vector unit
// is busy for 45 to 50% of it. 2000 x 4096 bf16 by columns 12.1 us, both ways 19;
// blocks of 12288 x 4096 fp32 both ways 54.5 us (302 MB, 5.5 TB/s).
template <typename TX>
__global__ __launch_bounds__(512) void k_fp8_tile(QuantFp8Args a, uint32_t blocks_k) {
  __shared__ float part[8][128];
  __shared__ Inverses inverses;
  __shared__ uint32_t cols[128 * Q_PITCH];
  const int l16 = threadIdx.x & 15, set = threadIdx.x >> 4, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t tile = blockIdx.x / blocks_k, g = blockIdx.x - tile * blocks_k;
  const int64_t r0 = (int64_t)tile * Q_ROWS, row = r0 + 4 * set, c0 = (int64_t)g * 128, col = c0 + 8 * l16;
  float v[4][8];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (row + r < a.m) {
      load_left((const TX*)a.x + (row + r) * a.ldx + col, a.k - col, v[r]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[r][j] = 0.f;
    }

  if (!a.blocks && a.q != nullptr) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float s = e4m3_scale(row_all<true>(max8(v[r])));
      const uint2 w = codes8(v[r], e4m3_inverse(s));
      if (row + r < a.m) {
        *reinterpret_cast<uint2*>(a.q + (row + r) * a.ldq + col) = w;
        if (l16 == 0) a.s[g * a.lds + row + r] = s;
      }
    }
  }

  // the scales of the tile's columns, or its one
  float m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = fmaxf(fmaxf(fabsf(v[0][j]), fabsf(v[1][j])), fmaxf(fabsf(v[2][j]), fabsf(v[3][j])));
    m[j] = rows_all<true>(m[j]);
  }
  if (a.blocks) {
    const float one = row_all<true>(max8(m));
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = one;
  }
  if (lane < 16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) part[wave][8 * l16 + j] = m[j];
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    float t = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) t = fmaxf(t, part[w][threadIdx.x]);
    const float s = e4m3_scale(t);
    inverses.put(threadIdx.x, e4m3_inverse(s));
    if (a.blocks) {
      if (threadIdx.x == 0) {
        if (a.q != nullptr) a.s[tile * a.lds + g] = s;
        if (a.qt != nullptr) a.st[g * a.ldst + tile] = s;
      }
    } else if (c0 + threadIdx.x < a.k) {
      a.st[tile * a.ldst + c0 + threadIdx.x] = s;
    }
  }
  __syncthreads();
  E4m3Inverse inv[8];
  bool slow = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    inv[j] = inverses.get(8 * l16 + j);
    slow |= inv[j].slow();
  }
  uint32_t w[4][2];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    e4m3_codes<8>(w[r], [&](int i) { return v[r][i]; }, [&](int i) { return (double)v[r][i]; },
                  [&](int i) { return inv[i]; }, slow);
    if (a.blocks && a.q != nullptr && row + r < a.m)
      *reinterpret_cast<uint2*>(a.q + (row + r) * a.ldq + col) = uint2{w[r][0], w[r][1]};
  }
  if (a.qt == nullptr) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t t[4];
    turn4(w[0][h], w[1][h], w[2][h], w[3][h], t);
#pragma unroll
    for (int j = 0; j < 4; ++j) cols[(8 * l16 + 4 * h + j) * Q_PITCH + set] = t[j];
  }
  __syncthreads();
  // eight lanes a column, 16 codes each
  for (int c = threadIdx.x >> 3; c < 128; c += 64) {
    const uint32_t* p = cols + c * Q_PITCH + 4 * (threadIdx.x & 7);
    if (c0 + c < a.k)
      *reinterpret_cast<u32x4_t*>(a.qt + (c0 + c) * a.ldqt + r0 + 16 * (threadIdx.x & 7)) =
          u32x4_t{p[0], p[1], p[2], p[3]};
  }
}

// ------------------------------------------------------------ rotated values
// A set of 16 lanes holds a 256-group of a row as 16 fp64 values each; after the
// transform register i of lane l is column 128 (l / 8) + l % 8 + 8 i of the
// group (row_sets.hpp), so a set's lanes 0 .. 7 hold its first block of 128.
namespace {

constexpr int Q_SET_BYTES = 16 * 18 * 8;

__device__ __forceinline__ int turned_col(int l16, int i) { return 128 * (l16 >> 3) + (l16 & 7) + 8 * i; }

template <typename TX>
__device__ __forceinline__ void rotated(const Runs<TX>& raw, double (&v)[16], uint8_t* buf, int l16) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = (double)raw.get(i) * 0.0625;
  fwht16_regs(v);
  transpose16(v, reinterpret_cast<double*>(buf), l16);
  fwht16_regs(v);
}

// Largest magnitude of the lane's block of 128.
__device__ __forceinline__ double half_set_max(double v) {
  v = fmax(v, swz_xor<1>(v));
  v = fmax(v, swz_xor<2>(v));
  v = fmax(v, swz_xor<4>(v));
  return v;
}

// The lane's 16 codes into the order of memory: 16 bytes of the group's row.
__device__ __forceinline__ u32x4_t straight(const uint32_t (&w)[4], uint8_t* buf, int l16) {
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < 16; ++i) buf[turned_col(l16, i)] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  wave_lds_sync();
  return *reinterpret_cast<const u32x4_t*>(buf + 16 * l16);
}

}  // namespace

// (4096 x 4096 bf16 16.7 us: fp64 on the vector unit, busy 60% of the time.)
template <typename TX>
__global__ __launch_bounds__(256) void k_fp8_rows_rotated(QuantFp8Args a, uint32_t groups) {
  __shared__ __align__(16) uint8_t turn[16 * Q_SET_BYTES];
  const int l16 = threadIdx.x & 15, set = threadIdx.x >> 4;
  const uint32_t tile = blockIdx.x / groups, g = blockIdx.x - tile * groups;
  const int64_t row = (int64_t)tile * 16 + set, c0 = (int64_t)g * 256;
  uint8_t* buf = turn + set * Q_SET_BYTES;
  Runs<TX> raw;
  if (row < a.m)
    raw.load((const TX*)a.x + row * a.ldx + c0 + 8 * l16);
  else
    raw.zero();
  double v[16];
  rotated(raw, v, buf, l16);
  const float s = e4m3_scale(half_set_max(absmax16(v)));
  const E4m3Inverse inv = e4m3_inverse(s);
  uint32_t w[4];
  e4m3_codes<16>(w, [&](int i) { return (float)v[i]; }, [&](int i) { return v[i]; }, [&](int) { return inv; },
                 inv.slow());
  const u32x4_t w4 = straight(w, buf, l16);
  if (row < a.m) {
    *reinterpret_cast<u32x4_t*>(a.q + row * a.ldq + c0 + 16 * l16) = w4;
    if ((l16 & 7) == 0) a.s[(2 * g + (l16 >> 3)) * a.lds + row] = s;
  }
}

// A tile of 128 rows and 256 columns, as k_fp8_tile; the four rows of a lane stay
// in registers as fp64 (two waves a SIMD; 2000 x 4096 bf16 by columns 15.4 us, the
// vector unit busy for a third of it: 256 blocks, one a compute unit).
template <typename TX>
__global__ __launch_bounds__(512, 2) void k_fp8_tile_rotated(QuantFp8Args a, uint32_t groups) {
  __shared__ __align__(16) uint8_t turn[32 * Q_SET_BYTES];
  __shared__ Inverses inverses;
  double(*part)[256] = reinterpret_cast<double(*)[256]>(turn);      // [8][256], after the transforms
  uint32_t* cols = reinterpret_cast<uint32_t*>(turn + 8 * 256 * 8);  // [256][Q_PITCH]
  static_assert(32 * Q_SET_BYTES >= 8 * 256 * 8 + 256 * Q_PITCH * 4, "the tile turns in the transforms' LDS");
  const int l16 = threadIdx.x & 15, set = threadIdx.x >> 4, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t tile = blockIdx.x / groups, g = blockIdx.x - tile * groups;
  const int64_t r0 = (int64_t)tile * Q_ROWS, row = r0 + 4 * set, c0 = (int64_t)g * 256;
  uint8_t* buf = turn + set * Q_SET_BYTES;
  Runs<TX> raw[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (row + r < a.m)
      raw[r].load((const TX*)a.x + (row + r) * a.ldx + c0 + 8 * l16);
    else
      raw[r].zero();
  double v[4][16];
#pragma unroll
  for (int r = 0; r < 4; ++r) rotated(raw[r], v[r], buf, l16);

  if (!a.blocks && a.q != nullptr) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float s = e4m3_scale(half_set_max(absmax16(v[r])));
      const E4m3Inverse inv = e4m3_inverse(s);
      uint32_t w[4];
      e4m3_codes<16>(w, [&](int i) { return (float)v[r][i]; }, [&](int i) { return v[r][i]; }, [&](int) { return inv; },
                     inv.slow());
      const u32x4_t w4 = straight(w, buf, l16);
      if (row + r < a.m) {
        *reinterpret_cast<u32x4_t*>(a.q + (row + r) * a.ldq + c0 + 16 * l16) = w4;
        if ((l16 & 7) == 0) a.s[(2 * g + (l16 >> 3)) * a.lds + row + r] = s;
      }
    }
  }
  __syncthreads();  // the transforms' LDS is free
  double m[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) m[i] = absmax2(absmax2(v[0][i], v[1][i]), absmax2(v[2][i], v[3][i]));
  if (a.blocks) {
    const double one = half_set_max(absmax16(m));
#pragma unroll
    for (int i = 0; i < 16; ++i) m[i] = one;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    m[i] = rows_all<true>(m[i]);
    if (lane < 16) part[wave][turned_col(l16, i)] = m[i];
  }
  __syncthreads();
  if (threadIdx.x < 256) {
    double t = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) t = fmax(t, part[w][threadIdx.x]);
    const float s = e4m3_scale(t);
    inverses.put(threadIdx.x, e4m3_inverse(s));
    if (a.blocks) {
      if ((threadIdx.x & 127) == 0) {
        const int64_t b = 2 * (int64_t)g + (threadIdx.x >> 7);
        if (a.q != nullptr) a.s[tile * a.lds + b] = s;
        if (a.qt != nullptr) a.st[b * a.ldst + tile] = s;
      }
    } else {
      a.st[tile * a.ldst + c0 + threadIdx.x] = s;
    }
  }
  __syncthreads();
  bool slow = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) slow |= inverses.get(turned_col(l16, i)).slow();
  uint32_t w[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    e4m3_codes<16>(w[r], [&](int i) { return (float)v[r][i]; }, [&](int i) { return v[r][i]; },
                   [&](int i) { return inverses.get(turned_col(l16, i)); }, slow);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t t[4];
    turn4(w[0][h], w[1][h], w[2][h], w[3][h], t);
#pragma unroll
    for (int j = 0; j < 4; ++j) cols[turned_col(l16, 4 * h + j) * Q_PITCH + set] = t[j];
  }
  __syncthreads();
  if (a.blocks && a.q != nullptr) {  // byte r of a column's dword is row 4 set + r
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t c = (cols[(16 * l16 + i) * Q_PITCH + set] >> (8 * r)) & 0xffu;
        w[i >> 2] = (i & 3) == 0 ? c : w[i >> 2] | (c << (8 * (i & 3)));
      }
      if (row + r < a.m)
        *reinterpret_cast<u32x4_t*>(a.q + (row + r) * a.ldq + c0 + 16 * l16) = u32x4_t{w[0], w[1], w[2], w[3]};
    }
  }
  if (a.qt == nullptr) return;
  for (int c = threadIdx.x >> 3; c < 256; c += 64) {
    const uint32_t* p = cols + c * Q_PITCH + 4 * (threadIdx.x & 7);
    *reinterpret_cast<u32x4_t*>(a.qt + (c0 + c) * a.ldqt + r0 + 16 * (threadIdx.x & 7)) = u32x4_t{p[0], p[1], p[2], p[3]};
  }
}

namespace {

template <typename TX>
hipError_t quant_launch(const QuantFp8Args& a, hipStream_t stream) {
  const bool tiles = a.blocks || a.qt != nullptr;
  const int64_t wide = a.rotate ? 256 : 128, high = tiles ? Q_ROWS : 16;
  const uint32_t bk = (uint32_t)((a.k + wide - 1) / wide);
  const dim3 grid((unsigned)((a.m + high - 1) / high * bk)), block(tiles ? 512 : 256);
  if (a.rotate) {
    if (tiles)
      hipLaunchKernelGGL((k_fp8_tile_rotated<TX>), grid, block, 0, stream, a, bk);
    else
      hipLaunchKernelGGL((k_fp8_rows_rotated<TX>), grid, block, 0, stream, a, bk);
  } else {
    if (tiles)
      hipLaunchKernelGGL((k_fp8_tile<TX>), grid, block, 0, stream, a, bk);
    else
      hipLaunchKernelGGL((k_fp8_rows<TX>), grid, block, 0, stream, a, bk);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(const QuantFp8Args& a, hipStream_t stream) {
  return a.x_bf16 ? quant_launch<uint16_t>(a, stream) : quant_launch<float>(a, stream);
}

}  // namespace tp
