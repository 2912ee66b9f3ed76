// The LoRA side path on activations kept in 8 bits, and its gradients
// (kvad-gpu internals, section "Pictures, which are not tokens": a side path
// (x.A).B beside a layer whose quantized weights stay as they are). The codes
// that the int8 product reads are also the checkpoint that the adapter's
// gradients are taken from: x[i] = sa[i] qa[i], in the rotated domain.
//
//  * down    T[i, j]  = sa[i] sum_q qa[i, q] A[j, q]
//  * dt      dT[i, j] = alpha sum_c dY[i, c] B[c, j]
//  * outer   dB[c, j] = alpha sum_i dY[i, c] T[i, j]
//            dA[j, q] = sum_i (dT[i, j] sa[i]) qa[i, q], rotated back on request
//
// All products run on bf16 matrix units with fp32 sums. Codes and bf16 values
// are exact bf16 operands; an fp32 operand is split exactly into three bf16
// parts (split3_bf16), and of two split operands the six products that reach
// above 2^-24 of the whole are taken: plain fp32 accuracy at 3 to 6 products.
// Long sums are split over blocks and joined in a fixed order (no atomics).
#include <type_traits>

#include "block_ops.hpp"
#include "device_common.hpp"
#include "group16.hpp"

namespace tp {

constexpr int SIDE_T = 64;   // floats of a row of T and dT (zeros past the rank)

// Sources of the streamed operand.
struct SrcBf16 { typedef uint16_t elem; static constexpr int PARTS = 1; };
struct SrcF32 { typedef float elem; static constexpr int PARTS = 3; };
struct SrcI8 { typedef int8_t elem; static constexpr int PARTS = 1; };

__device__ __forceinline__ bf16x8_t as_bf16(u32x4_t w) { return __builtin_bit_cast(bf16x8_t, w); }

// 8 codes (exact in bf16).
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi) {
  u32x4_t w;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    w[p] = pack_bf16x2((float)(int8_t)(lo >> (16 * p)), (float)(int8_t)(lo >> (16 * p + 8)));
    w[2 + p] = pack_bf16x2((float)(int8_t)(hi >> (16 * p)), (float)(int8_t)(hi >> (16 * p + 8)));
  }
  return as_bf16(w);
}

// acc += the products of two operands in parts (part 0 the largest); parts
// whose product is below 2^-24 of the whole are left out.
template <int PX, int PY>
__device__ __forceinline__ f32x4_t mfma_parts(const bf16x8_t (&x)[PX], const bf16x8_t (&y)[PY], f32x4_t acc) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < PX; ++i)
#pragma unroll
      for (int j = 0; j < PY; ++j)
        if (i + j == s) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y[j], acc, 0, 0, 0);
  return acc;
}

// 8 consecutive elements of a row as an operand in parts; `valid` of them are
// read, the others are zero.
__device__ __forceinline__ void load_parts(const uint16_t* p, int valid, bf16x8_t (&o)[1]) {
  u32x4_t w = {0u, 0u, 0u, 0u};
  if (valid >= 8) {
    w = *reinterpret_cast<const u32x4_t*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  }
  o[0] = as_bf16(w);
}

__device__ __forceinline__ void load_f32x8(const float* p, int valid, float (&v)[8]) {
  if (valid >= 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < valid ? p[e] : 0.f;
  }
}

__device__ __forceinline__ void load_parts(const float* p, int valid, bf16x8_t (&o)[3]) {
  float v[8];
  load_f32x8(p, valid, v);
  split3_bf16(v, o[0], o[1], o[2]);
}

// 8 consecutive elements as loaded, and as an operand.
template <typename T> struct RawOp;

template <> struct RawOp<uint16_t> {
  u32x4_t w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const u32x4_t*>(p); }
  __device__ __forceinline__ void load(const uint16_t* p, int valid) {
    bf16x8_t o[1];
    load_parts(p, valid, o);
    w = __builtin_bit_cast(u32x4_t, o[0]);
  }
  __device__ __forceinline__ void parts(bf16x8_t (&o)[1]) const { o[0] = as_bf16(w); }
};

template <> struct RawOp<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void load(const float* p, int valid) { load_f32x8(p, valid, v); }
  __device__ __forceinline__ void parts(bf16x8_t (&o)[3]) const { split3_bf16(v, o[0], o[1], o[2]); }
};

// --------------------------------------------------------------------- down
// Partial sums of qa . A^T: a block owns 16 WR FM rows and a run of 256-column
// chunks of A, which its waves share through LDS (A read by every 16 rows from
// memory made one compute unit's loads the bound: 24 us for a single row of
// 12288 columns at rank 32). Lane l feeds row l % 16 with the 16 codes
// 16 (l / 16) of each 64; A's columns are stored in the order in which the two
// products of a step take them. With few rows (WR 1) the waves share a chunk and
// join their sums in LDS (one row of 12288 columns at rank 16: 12.8 us with the
// join over blocks, 17.3 with a partial sum a wave and no limit on the splits).
// 4096 x 12288 at rank 32: 14.4 us (3.6 TB/s; two to three chunks a block).
constexpr int SD_KC = 256;  // columns per chunk of the plan

// Columns in LDS at a time: half a chunk where 64 ranks of an fp32 A (three planes,
// 101 KiB) would leave one block a compute unit (4096 x 12288: 30 us, 40 with
// whole chunks). A row's pitch is 8 more: rows 4 banks apart.
template <typename TA, int R, int WR>
constexpr int down_columns() {
  return std::is_same<TA, float>::value && R == 64 && WR == 4 ? SD_KC / 2 : SD_KC;
}

struct DownArgs {
  const int8_t* qa;
  int64_t ldqa;
  const void* a;
  int64_t lda, m;
  int r, splits, chunks_per_split, chunks;
  float* part;  // [splits, m, R]
};

template <typename TA, int R, int WR, int FM>
__global__ __launch_bounds__(256, (std::is_same<TA, float>::value && R == 64 && WR == 1) ? 1 : 2)  //
    void k_side_down(DownArgs d) {
  constexpr int NF = R / 16;
  constexpr int PA = std::is_same<TA, float>::value ? 3 : 1;
  constexpr int WN = 4 / WR;
  constexpr int KC = down_columns<TA, R, WR>(), PITCH = KC + 8;
  constexpr int STEPS = KC / 64 / WN;        // 64-column steps of a wave and chunk
  constexpr int PLANE = R * PITCH;
  constexpr int RUNS = KC / 8, RANKS = 256 / RUNS;  // runs of 8 columns, and ranks that the threads stage at a time
  constexpr int UNITS = R / RANKS;                  // runs that a thread stages
  __shared__ __align__(16) uint16_t at[PA * PLANE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int rg = wave % WR, ns = wave / WR;
  const int split = (int)(blockIdx.x % (unsigned)d.splits);
  const int64_t m0 = ((int64_t)(blockIdx.x / (unsigned)d.splits) * WR + rg) * (16 * FM);
  const int c0 = split * d.chunks_per_split * (SD_KC / KC);
  const int c1 = min(c0 + d.chunks_per_split * (SD_KC / KC), d.chunks * (SD_KC / KC));
  // Rows past the last one and ranks past r read the last row or rank instead:
  // what comes of them is not written.
  const int8_t* xrow[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i)
    xrow[i] = d.qa + min(m0 + 16 * i + l16, d.m - 1) * d.ldqa + ns * (64 * STEPS) + 16 * g4;
  const int ar = threadIdx.x / RUNS, ak = threadIdx.x % RUNS;  // rank (of RANKS at a time) and run of 8 columns staged
  u32x4_t x[FM][STEPS];
  RawOp<TA> av[UNITS];
  auto load_x = [&](int c) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        x[i][s] = *reinterpret_cast<const u32x4_t*>(xrow[i] + (int64_t)c * KC + 64 * s);
  };
  auto load_a = [&](int c) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      av[u].load((const TA*)d.a + (int64_t)min(ar + RANKS * u, d.r - 1) * d.lda + (int64_t)c * KC + 8 * ak);
  };
  f32x4_t acc[FM][NF];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[i][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (c0 < c1) {
    load_a(c0);
    load_x(c0);
  }
  // columns 64 s + 16 g + 8 h of a chunk sit at 64 s + 32 h + 8 g
  const int pos = (ak >> 3) * 64 + (ak & 1) * 32 + ((ak >> 1) & 3) * 8;
  for (int c = c0; c < c1; ++c) {
    __syncthreads();
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      bf16x8_t o[PA];
      av[u].parts(o);
#pragma unroll
      for (int p = 0; p < PA; ++p)
        *reinterpret_cast<bf16x8_t*>(at + p * PLANE + (ar + RANKS * u) * PITCH + pos) = o[p];
    }
    __syncthreads();
    u32x4_t now[FM][STEPS];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) now[i][s] = x[i][s];
    if (c + 1 < c1) {
      load_a(c + 1);
      load_x(c + 1);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bf16x8_t xp[FM][1];
#pragma unroll
        for (int i = 0; i < FM; ++i)
          xp[i][0] = h ? widen8(now[i][s].z, now[i][s].w) : widen8(now[i][s].x, now[i][s].y);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          bf16x8_t ap[PA];
#pragma unroll
          for (int p = 0; p < PA; ++p)
            ap[p] = *reinterpret_cast<const bf16x8_t*>(at + p * PLANE + (16 * f + l16) * PITCH +
                                                       64 * (ns * STEPS + s) + 32 * h + 8 * g4);
#pragma unroll
          for (int i = 0; i < FM; ++i) acc[i][f] = mfma_parts(xp[i], ap, acc[i][f]);
        }
      }
  }
  if constexpr (WN > 1) {  // the waves' sums of the same rows, added in wave order
    float* red = reinterpret_cast<float*>(at);
    static_assert(FM == 1 && WN * 16 * R * 4 <= PA * PLANE * 2, "the sums fit in the staging area");
    __syncthreads();
#pragma unroll
    for (int f = 0; f < NF; ++f) *reinterpret_cast<f32x4_t*>(red + ((wave * NF + f) * 64 + lane) * 4) = acc[0][f];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < WN; ++w)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[0][f] += *reinterpret_cast<const f32x4_t*>(red + ((w * NF + f) * 64 + lane) * 4);
  }
  // lane l holds rows 4 (l / 16) + v, column 16 f + l % 16
  float* out = d.part + (int64_t)split * d.m * R;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t row = m0 + 16 * i + 4 * g4 + v;
      if (row < d.m) {
#pragma unroll
        for (int f = 0; f < NF; ++f) out[row * R + 16 * f + l16] = acc[i][f][v];
      }
    }
}

// ----------------------------------------------------------------------- dt
// Partial sums of dY . B: a block owns 16 WR rows and a run of 256-column
// chunks; the chunk of B is transposed (and split) into LDS, from where it is
// the matrix units' second operand, and dY goes straight from memory to the
// first. With few rows (WR 1) the four waves share the chunk instead. 4096 x 9216
// bf16 at rank 32: 17.0 us (4.6 TB/s).
constexpr int DT_NC = 256;  // columns of dY per chunk of the plan

// Columns in LDS at a time: half a chunk of an fp32 B's three planes, from 32
// ranks on: with 50 and 101 KiB fewer blocks share a compute unit (4096 x 9216
// bf16 at rank 64: 30 us, 51 with whole chunks that half of the threads stage; at
// rank 32 20 and 25). A row's pitch is 8 more: rows 4 banks apart.
template <typename TB, int R>
constexpr int dt_columns() {
  return std::is_same<TB, float>::value && R >= 32 ? DT_NC / 2 : DT_NC;
}

// Two dwords' low (odd == 0) or high halves in one.
__device__ __forceinline__ uint32_t pair_of(uint32_t first, uint32_t second, int odd) {
  return __builtin_amdgcn_perm(second, first, odd ? 0x07060302u : 0x05040100u);
}

// 8 x W elements of a lane (row i, column c), and column c as an operand of
// the 8 rows: 16-bit halves are paired by byte permutes, fp32 columns split.
template <typename SRC, int W = 8> struct Block8;

template <> struct Block8<SrcBf16, 8> {
  u32x4_t w[8];
  __device__ __forceinline__ void zero(int i) { w[i] = u32x4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void load(int i, const uint16_t* p) { w[i] = *reinterpret_cast<const u32x4_t*>(p); }
  __device__ __forceinline__ void load(int i, const uint16_t* p, int valid) {
    bf16x8_t o[1];
    load_parts(p, valid, o);
    w[i] = __builtin_bit_cast(u32x4_t, o[0]);
  }
  __device__ __forceinline__ void column(int c, bf16x8_t (&o)[1]) const {
    u32x4_t v;
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = pair_of(w[2 * p][c >> 1], w[2 * p + 1][c >> 1], c & 1);
    o[0] = as_bf16(v);
  }
};

template <int W> struct Block8<SrcF32, W> {
  typedef float run_t __attribute__((ext_vector_type(W < 4 ? W : 4)));
  static constexpr int RUN = W < 4 ? W : 4;
  float w[8][W];
  __device__ __forceinline__ void zero(int i) {
#pragma unroll
    for (int c = 0; c < W; ++c) w[i][c] = 0.f;
  }
  __device__ __forceinline__ void load(int i, const float* p) {
#pragma unroll
    for (int c = 0; c < W; c += RUN) {
      const run_t v = *reinterpret_cast<const run_t*>(p + c);
#pragma unroll
      for (int e = 0; e < RUN; ++e) w[i][c + e] = v[e];
    }
  }
  __device__ __forceinline__ void load(int i, const float* p, int valid) {
    if (valid >= W) {
      load(i, p);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) w[i][e] = e < valid ? p[e] : 0.f;
    }
  }
  __device__ __forceinline__ void column(int c, bf16x8_t (&o)[3]) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i][c];
    split3_bf16(v, o[0], o[1], o[2]);
  }
};

template <> struct Block8<SrcI8, 8> {
  uint2 w[8];
  __device__ __forceinline__ void zero(int i) { w[i] = uint2{0u, 0u}; }
  __device__ __forceinline__ void load(int i, const int8_t* p) { w[i] = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void load(int i, const int8_t* p, int valid) {  // k is a multiple of 256: all 8 or none
    if (valid > 0)
      load(i, p);
    else
      zero(i);
  }
  __device__ __forceinline__ void column(int c, bf16x8_t (&o)[1]) const {
    u32x4_t v;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t a = c < 4 ? w[2 * p].x : w[2 * p].y, b = c < 4 ? w[2 * p + 1].x : w[2 * p + 1].y;
      v[p] = pack_bf16x2((float)(int8_t)(a >> (8 * (c & 3))), (float)(int8_t)(b >> (8 * (c & 3))));
    }
    o[0] = as_bf16(v);
  }
};

struct DtArgs {
  const void* dy;
  int64_t lddy;
  const void* b;
  int64_t ldb, m, n;
  int r, splits, chunks_per_split;
  float* part;  // [splits, m, R]
};

// The next chunk's dY and B are in flight while a chunk is multiplied; only B
// where an fp32 dY's registers would leave one block less a compute unit (fp32 dY
// and B, 4096 x 9216: 36 us with it and 40 without at rank 32, 56 and 48 at 64).
template <typename SRC, typename TB, int R, int WR>
__device__ __forceinline__ void dt_block(const DtArgs& a, unsigned blk, uint16_t* bt) {
  typedef typename SRC::elem TY;
  typedef typename std::conditional<std::is_same<TB, float>::value, SrcF32, SrcBf16>::type BSRC;
  constexpr int NF = R / 16;
  constexpr int PY = SRC::PARTS, PB = BSRC::PARTS;
  constexpr int NC = dt_columns<TB, R>(), PITCH = NC + 8;
  constexpr int WN = 4 / WR;             // waves that share a chunk
  constexpr int STEPS = NC / 32 / WN;    // 32-column steps of a wave and chunk
  constexpr int PLANE = R * PITCH;
  constexpr bool AHEAD = PY == 1 || (NC < DT_NC && R < 64);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int rg = wave % WR, ns = wave / WR;
  const int split = (int)(blk % (unsigned)a.splits);
  const int64_t m0 = (int64_t)(blk / (unsigned)a.splits) * (16 * WR) + 16 * rg;
  // rows past the last one read that one: what comes of them is not written
  const TY* row = (const TY*)a.dy + min(m0 + l16, a.m - 1) * a.lddy + ns * (32 * STEPS) + 8 * g4;
  const int64_t nchunks = (a.n + NC - 1) / NC;
  const int per_split = a.chunks_per_split * (DT_NC / NC);
  const int64_t c0 = (int64_t)split * per_split, c1 = min(c0 + per_split, nchunks);
  // This thread's block of a chunk of B: 8 columns, 8 ranks of a bf16 B; of an fp32
  // B, which costs a split into three parts, as few as give every thread one.
  constexpr int W = PB == 1 ? 8 : R * NC / 8 / 256;
  const int nb = threadIdx.x / (R / W), jb = threadIdx.x % (R / W);
  const bool stages = nb < NC / 8;
  const int cols = max(0, min(W, a.r - W * jb));
  const TB* bcol = (const TB*)a.b + (cols > 0 ? W * jb : 0);

  // Where a run of 8 columns stands in an LDS row: its number, exclusive or the
  // rank / 8, so that the runs that a wave stores at a time fall on different banks.
  const int swz[2] = {8 * (g4 ^ (l16 >> 3)), 8 * (g4 ^ (2 + (l16 >> 3)))};

  RawOp<TY> y[STEPS];
  Block8<BSRC, W> bb;
  auto load_y = [&](int64_t c) {
    const int64_t n0 = c * NC;
    if (n0 + NC <= a.n) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) y[s].load(row + n0 + 32 * s);
    } else {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int64_t left = a.n - (n0 + ns * (32 * STEPS) + 32 * s + 8 * g4);
        y[s].load(left > 0 ? row + n0 + 32 * s : row, (int)max((int64_t)0, min((int64_t)8, left)));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  auto load_b = [&](int64_t c) {
    if (!stages) return;
    const int64_t n = c * NC + 8 * nb;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (n + i < a.n)
        bb.load(i, bcol + (n + i) * a.ldb, cols);
      else
        bb.zero(i);
    }
  };
  f32x4_t acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (c0 < c1) {
    load_b(c0);
    if (AHEAD) load_y(c0);
  }
  for (int64_t c = c0; c < c1; ++c) {
    if (!AHEAD) load_y(c);
    __syncthreads();
    if (stages) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        bf16x8_t o[PB];
        bb.column(e, o);
#pragma unroll
        for (int p = 0; p < PB; ++p)
          *reinterpret_cast<bf16x8_t*>(bt + p * PLANE + (W * jb + e) * PITCH + 8 * (nb ^ (W * jb >> 3))) = o[p];
      }
    }
    __syncthreads();
    RawOp<TY> now[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) now[s] = y[s];
    if (c + 1 < c1) {
      load_b(c + 1);
      if (AHEAD) load_y(c + 1);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      bf16x8_t yp[PY];
      now[s].parts(yp);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        bf16x8_t bp[PB];
#pragma unroll
        for (int p = 0; p < PB; ++p)
          bp[p] = *reinterpret_cast<const bf16x8_t*>(bt + p * PLANE + (16 * f + l16) * PITCH +
                                                     32 * ((ns * STEPS + s) ^ (f >> 1)) + swz[f & 1]);
        acc[f] = mfma_parts(yp, bp, acc[f]);
      }
    }
  }
  if constexpr (WN > 1) {  // the waves' sums of the same rows, added in wave order
    float* red = reinterpret_cast<float*>(bt);
    static_assert(WN * 16 * R * 4 <= PB * PLANE * 2, "the sums fit in the staging area");
    __syncthreads();
#pragma unroll
    for (int f = 0; f < NF; ++f) *reinterpret_cast<f32x4_t*>(red + ((wave * NF + f) * 64 + lane) * 4) = acc[f];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < WN; ++w)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[f] += *reinterpret_cast<const f32x4_t*>(red + ((w * NF + f) * 64 + lane) * 4);
  }
  float* out = a.part + ((int64_t)split * a.m + m0) * R;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (m0 + 4 * g4 + v < a.m) {
#pragma unroll
      for (int f = 0; f < NF; ++f) out[(int64_t)(4 * g4 + v) * R + 16 * f + l16] = acc[f][v];
    }
}

// -------------------------------------------------------------------- outer
// Partial sums over rows of small^T . big: small [rows, r] (T, or dT sa) as
// three bf16 parts in planes of 32-row chunks (k_side_prep), big [rows, width]
// streamed from memory. The sum runs over the rows, so a lane loads an 8 x 8
// block (8 rows, 8 columns): its column c is an operand of 8 consecutive rows,
// and 16 lanes cover 128 columns, every eighth at a time. A block owns 128
// columns, up to 32 ranks and a run of chunks, which its four waves take in
// turn; their sums are added in LDS in wave order. The next chunk is in flight
// while one is multiplied; bound by that chain of loads (4096 x 9216 bf16 and 4096
// x 3072 codes at rank 32: 20.5 us; dB alone 17.6, of which its loads take 16.7).
constexpr int OU_MC = 32;     // rows per chunk
constexpr int OU_COLS = 128;  // columns of a block
constexpr int OU_RB = 32;     // ranks of a block, at most

struct OuterArgs {
  const void* big;
  int64_t ldbig, width;   // [m, width]
  const uint16_t* small;  // planes [3, nmc, R, 32]
  int64_t m;
  int splits, chunks_per_split;
  int64_t nmc;            // 32-row chunks
  float* part;            // [splits, width, R]; of codes: [splits, R, width]
};

template <int R> struct OuterShape {
  static constexpr int RB = R < OU_RB ? R : OU_RB;  // ranks of a block
  static constexpr int HALVES = R / RB;
  static unsigned blocks(int64_t units) { return (unsigned)(HALVES > 1 ? (units + 7) / 8 * 8 * HALVES : units); }
  static constexpr int LDS = 4 * 2 * (RB / 16) * 64;  // f32x4: two columns' sums of four waves
};

template <typename SRC, int R, bool BY_RANK>
__device__ __forceinline__ void outer_block(const OuterArgs& a, unsigned blk, f32x4_t* red) {
  typedef typename SRC::elem TY;
  constexpr int RB = OuterShape<R>::RB, HALVES = OuterShape<R>::HALVES;
  constexpr int NF = RB / 16, PS = SRC::PARTS;
  constexpr bool AHEAD = PS == 1;  // fp32 columns leave no registers for a second block
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g4 = lane >> 4;
  // Blocks go to the eight XCDs in turn: the halves of the ranks, which read the
  // same columns, are eight apart, so that one L2 serves both (4096 x 9216 bf16 at
  // rank 64: 30.0 us, 35.8 as neighbours).
  const int j0 = HALVES > 1 ? (int)(blk / 8 % HALVES) * RB : 0;
  const unsigned unit = HALVES > 1 ? blk / (8 * HALVES) * 8 + blk % 8 : blk;
  const int split = (int)(unit % (unsigned)a.splits);
  const int64_t col0 = (int64_t)(unit / (unsigned)a.splits) * OU_COLS, col = col0 + 8 * l16;
  if (col0 >= a.width) return;  // (the units are made up to a multiple of eight)
  const int valid = (int)max((int64_t)0, min((int64_t)8, a.width - col));
  const bool inside = col0 + OU_COLS <= a.width;
  const TY* big = (const TY*)a.big + (valid > 0 ? col : 0);
  const uint16_t* small = a.small + (j0 + l16) * OU_MC + 8 * g4;
  const int64_t plane = a.nmc * (R * OU_MC);
  const int64_t c0 = (int64_t)split * a.chunks_per_split, c1 = min(c0 + a.chunks_per_split, a.nmc);
  f32x4_t acc[8][NF];
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[c][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  bf16x8_t sm[NF][3];
  auto load_small = [&](int64_t ch) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int p = 0; p < 3; ++p)
        sm[f][p] = *reinterpret_cast<const bf16x8_t*>(small + p * plane + ch * (R * OU_MC) + f * (16 * OU_MC));
  };
  auto load_big = [&](int64_t ch, Block8<SRC>& b) {
    const int64_t r0 = ch * OU_MC;
    if (inside && r0 + OU_MC <= a.m) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b.load(i, big + (r0 + 8 * g4 + i) * a.ldbig);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + 8 * g4 + i;
        if (row < a.m)
          b.load(i, big + row * a.ldbig, valid);
        else
          b.zero(i);
        __builtin_amdgcn_sched_barrier(0);  // one row's elements at a time: the edges need no more registers
      }
    }
  };
  Block8<SRC> next;
  int64_t ch = c0 + wave;
  if (ch < c1) {
    load_small(ch);
    if (AHEAD) load_big(ch, next);
  }
  for (; ch < c1; ch += 4) {
    if (!AHEAD) load_big(ch, next);
    const Block8<SRC> now = next;
    bf16x8_t sn[NF][3];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int p = 0; p < 3; ++p) sn[f][p] = sm[f][p];
    if (ch + 4 < c1) {
      load_small(ch + 4);
      if (AHEAD) load_big(ch + 4, next);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      bf16x8_t bc[PS];
      now.column(c, bc);
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[c][f] = mfma_parts(sn[f], bc, acc[c][f]);
      if (c & 1) __builtin_amdgcn_sched_barrier(0);  // two columns' operands at a time
    }
  }
  // lane l holds, for column col + c, the ranks j0 + 16 f + 4 (l / 16) + v. Two
  // columns' sums at a time (c and c + 4) go through LDS, where a thread adds
  // the waves' sums of one: four columns in a row after the four rounds.
  // red: [wave][column][f][lane]
  const int half = (int)threadIdx.x / (64 * NF), f = (int)threadIdx.x / 64 % NF;
  f32x4_t sum[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = 0; g < NF; ++g) red[((wave * 2 + h) * NF + g) * 64 + lane] = acc[c + 4 * h][g];
    __syncthreads();
    if (half < 2) {
      sum[c] = red[(half * NF + f) * 64 + lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) sum[c] += red[((w * 2 + half) * NF + f) * 64 + lane];
    }
  }
  if (half >= 2) return;
  const int j = j0 + 16 * f + 4 * g4;
  if constexpr (BY_RANK) {  // [splits, R, width]; the width is a multiple of 256
#pragma unroll
    for (int v = 0; v < 4; ++v)
      *reinterpret_cast<f32x4_t*>(a.part + ((int64_t)split * R + j + v) * a.width + col + 4 * half) =
          f32x4_t{sum[0][v], sum[1][v], sum[2][v], sum[3][v]};
  } else {  // [splits, width, R]
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (4 * half + c < valid)
        *reinterpret_cast<f32x4_t*>(a.part + ((int64_t)split * a.width + col + 4 * half + c) * R + j) = sum[c];
  }
}

template <typename SRC, typename TB, int R, int WR>
__global__ __launch_bounds__(256) void k_side_dt(DtArgs t) {
  constexpr int PB = std::is_same<TB, float>::value ? 3 : 1;
  __shared__ __align__(16) uint16_t lds[PB * R * (dt_columns<TB, R>() + 8)];
  dt_block<SRC, TB, R, WR>(t, blockIdx.x, lds);
}

// dB's sums and dA's in one launch: the first nb_db blocks take dB's, the others
// dA's (which alone do not fill the chip).
template <typename SRC, int R>
__global__ __launch_bounds__(256) void k_side_outer(OuterArgs db, OuterArgs da, unsigned nb_db) {
  __shared__ f32x4_t red[OuterShape<R>::LDS];
  if (blockIdx.x < nb_db)
    outer_block<SRC, R, false>(db, blockIdx.x, red);
  else
    outer_block<SrcI8, R, true>(da, blockIdx.x - nb_db, red);
}

// --------------------------------------------------------------------- join
// The sum of `splits` partial sums, `pitch` floats apart, in order: eight loads
// in flight, the last ones clamped.
__device__ __forceinline__ f32x4_t sum_splits(const float* p, int64_t pitch, int splits) {
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  for (int q0 = 0; q0 < splits; q0 += 8) {
    f32x4_t w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = *reinterpret_cast<const f32x4_t*>(p + min(q0 + q, splits - 1) * pitch);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q0 + q < splits) s += w[q];
  }
  return s;
}

// T: the splits added in order, four ranks a thread, times the rows' factors:
// rows of 64, zeros past the rank.
template <int R>
__global__ __launch_bounds__(256) void k_side_join_t(const float* __restrict__ p, int splits, int64_t M,
                                                     const float* __restrict__ rowscale, int r,
                                                     float* __restrict__ t) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, row = e / (SIDE_T / 4);
  const int j = (int)(e % (SIDE_T / 4)) * 4;
  if (row >= M) return;
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  if (j < r) {
    s = sum_splits(p + row * R + j, M * R, splits) * rowscale[row];
#pragma unroll
    for (int v = 0; v < 4; ++v) s[v] = j + v < r ? s[v] : 0.f;
  }
  *reinterpret_cast<f32x4_t*>(t + row * SIDE_T + j) = s;
}

// The small operands of the outer products, one 32-row chunk a block: the first
// nmc blocks add dT's splits in order, times alpha, into dt (rows of 64, zeros
// past the rank), and split dT sa into planes; the others split T. Rows past
// the last one and ranks past r are zeros in the planes.
template <int R>
__global__ __launch_bounds__(512) void k_side_prep(const float* __restrict__ part, int splits, int64_t M,
                                                   const float* __restrict__ sa, float alpha, int r,
                                                   const float* __restrict__ t, float* __restrict__ dt,
                                                   uint16_t* __restrict__ dt_planes,
                                                   uint16_t* __restrict__ t_planes, int64_t nmc) {
  __shared__ float tile[OU_MC][R + 1];
  const bool is_dt = (int64_t)blockIdx.x < nmc;
  const int64_t ch = is_dt ? blockIdx.x : blockIdx.x - nmc;
  {
    const int i = threadIdx.x / (SIDE_T / 4), j = threadIdx.x % (SIDE_T / 4) * 4;  // 32 rows of 16 quads
    const int64_t row = ch * OU_MC + i;
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
    if (row < M && j < r) {
      s = is_dt ? sum_splits(part + row * R + j, M * R, splits) * alpha
                : *reinterpret_cast<const f32x4_t*>(t + row * SIDE_T + j);
#pragma unroll
      for (int v = 0; v < 4; ++v) s[v] = j + v < r ? s[v] : 0.f;
    }
    if (is_dt && row < M) {
      *reinterpret_cast<f32x4_t*>(dt + row * SIDE_T + j) = s;
      s = s * sa[row];
    }
    if (j < R) {
#pragma unroll
      for (int v = 0; v < 4; ++v) tile[i][j + v] = s[v];
    }
  }
  __syncthreads();
  uint16_t* planes = is_dt ? dt_planes : t_planes;
  const int64_t plane = nmc * (R * OU_MC);
  if (threadIdx.x < R * (OU_MC / 8)) {
    const int j = threadIdx.x % R, oct = threadIdx.x / R;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = tile[8 * oct + i][j];
    bf16x8_t h, m, l;
    split3_bf16(v, h, m, l);
    uint16_t* to = planes + (ch * R + j) * OU_MC + 8 * oct;
    *reinterpret_cast<bf16x8_t*>(to) = h;
    *reinterpret_cast<bf16x8_t*>(to + plane) = m;
    *reinterpret_cast<bf16x8_t*>(to + 2 * plane) = l;
  }
}

// The splits of dB [splits, N, R] and dA [splits, R, K] added. The first nb_db
// blocks take dB, four ranks a thread, times alpha. In the others a half wave
// takes every fourth split of a 256-group of one rank of dA, eight of these
// units a block; the four sums are joined in LDS, and the first half wave of a
// unit rotates the group back on request.
template <int R>
__global__ __launch_bounds__(1024) void k_side_join(const float* __restrict__ pb, int sb, int64_t N,
                                                    float* __restrict__ db, int64_t lddb, float alpha,
                                                    const float* __restrict__ pa, int splits, int K,
                                                    float* __restrict__ da, int64_t ldda, int rotate, int r,
                                                    unsigned nb_db) {
  __shared__ __align__(16) float sums[4][8][256];
  if (blockIdx.x < nb_db) {
    const int64_t e = (int64_t)blockIdx.x * 1024 + threadIdx.x, row = e / (R / 4);
    const int j = (int)(e % (R / 4)) * 4;
    if (row >= N || j >= r) return;
    const f32x4_t s = sum_splits(pb + row * R + j, N * R, sb);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (j + v < r) db[row * lddb + j + v] = s[v] * alpha;
    return;
  }
  const int lane32 = threadIdx.x & 31, i = (threadIdx.x >> 5) & 7, part = threadIdx.x >> 8;
  const int groups = K / 256, units = r * groups;
  const int unit = (int)(blockIdx.x - nb_db) * 8 + i;
  const int j = unit / groups, c = (unit - j * groups) * 256 + lane32 * 8;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
  if (unit < units) {
    for (int q0 = part; q0 < splits; q0 += 16) {  // four splits in flight, the last ones clamped
      float w[4][8];
#pragma unroll
      for (int q = 0; q < 4; ++q) load8(pa + ((int64_t)min(q0 + 4 * q, splits - 1) * R + j) * K + c, w[q]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q0 + 4 * q < splits) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += w[q][e];
        }
    }
  }
  store8(&sums[part][i][8 * lane32], v);
  __syncthreads();
  if (part != 0 || unit >= units) return;  // uniform over the half wave that owns the unit
#pragma unroll
  for (int q = 1; q < 4; ++q) {
    float w[8];
    load8(&sums[q][i][8 * lane32], w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
  }
  if (rotate) {
    fwht256_lane8(v, lane32);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= 0.0625f;
  }
  store8(da + (int64_t)j * ldda + c, v);
}

// ---------------------------------------------------------------- launchers
namespace {

// How the sums are split: enough blocks for the chip, as few partial sums as
// that allows. Up to 16 rows a block's waves share a chunk, beyond that each takes
// 16 rows: whole gradients of 8 rows 15.9 us at n 9216, k 3072, rank 32 (16.3 with
// 64-row blocks), 14.0 at n 1160, k 1280, rank 8, fp32 (15.4). The border stands where
// 16-row blocks begin to read B twice; up to 64 rows they would still be the faster
// ones by 0.6 to 1.4 us (64 rows: 17.6 and 18.2 us, at n 1160 15.0 and 16.4).
// dT's target of 768 blocks, 512 and 1024 beside it: 4096 rows bf16 49.6 us, 49.3,
// 49.6; all fp32 at rank 64 113.0, 116.7, 112.9; an fp32 B at rank 64 71.1, 76.1, 71.0.
struct SidePlan {
  int wr;                        // row groups of a dt block
  int64_t rb, nchunks;           // row blocks, 256-column chunks (dt)
  int s1, cps1;                  // splits of the columns, chunks of a split
  int64_t nmc;                   // 32-row chunks (outer)
  int64_t cb2, cb3;              // column blocks of dB and dA
  int s2, cps2, s3, cps3;
  int64_t off2, off3;            // floats: the dB and dA partial sums
  int64_t off4, off5, total;     // the planes of dT sa and of T, and all
};

int padded_rank(int64_t r) { return r <= 16 ? 16 : r <= 32 ? 32 : 64; }

void split_of(int64_t chunks, int64_t want, int* splits, int* per) {
  if (chunks == 0) {
    *splits = 0;
    *per = 0;
    return;
  }
  const int64_t s = want < 1 ? 1 : (want > chunks ? chunks : want);
  const int64_t p = (chunks + s - 1) / s;
  *per = (int)p;
  *splits = (int)((chunks + p - 1) / p);
}

SidePlan side_plan(int64_t m, int64_t n, int64_t k, int64_t r) {
  SidePlan p;
  const int R = padded_rank(r);
  p.wr = m > 16 ? 4 : 1;
  p.rb = (m + 16 * p.wr - 1) / (16 * p.wr);
  p.nchunks = (n + DT_NC - 1) / DT_NC;
  const int64_t want1 = p.rb > 0 ? 768 / p.rb : 0;
  split_of(m > 0 ? p.nchunks : 0, want1 < 24 ? want1 : 24, &p.s1, &p.cps1);  // (as in down_plan)
  p.nmc = (m + OU_MC - 1) / OU_MC;
  p.cb2 = (n + OU_COLS - 1) / OU_COLS;
  p.cb3 = (k + OU_COLS - 1) / OU_COLS;
  // Two blocks a compute unit are resident: dB's and dA's together are made to
  // fit in that once (4096 rows bf16 49.6 us; 48.5 with 256 blocks and 51.2 with
  // 1024; fp32 dY at 3072 columns and rank 16 34.3, 36.2, 36.7; all fp32 at rank 64 and
  // 2048 rows 70.2, 75.7, 70.1). A split is at least a chunk for each of the four waves.
  const int64_t quads = (p.nmc + 3) / 4, want = 512 / ((p.cb2 + p.cb3) * (R > OU_RB ? R / OU_RB : 1));
  split_of(n > 0 ? quads : 0, want, &p.s2, &p.cps2);
  split_of(quads, want, &p.s3, &p.cps3);
  p.cps2 *= 4;
  p.cps3 *= 4;
  p.off2 = (int64_t)p.s1 * m * R;
  p.off3 = p.off2 + (int64_t)p.s2 * n * R;
  p.off4 = p.off3 + (int64_t)p.s3 * k * R;
  const int64_t planes = 3 * p.nmc * R * OU_MC / 2;  // in floats
  p.off5 = p.off4 + planes;
  p.total = p.off5 + planes;
  return p;
}

struct DownPlan {
  int wr, fm;
  int64_t rb;
  int s, cps;
  int64_t total;  // floats
};

// Up to 16 rows the waves of a block share a chunk (one row of 12288 columns at rank
// 32 5.5 us, 6.0 with 64-row blocks; 16 rows 6.4, 7.0; 17 to 64 rows would take 0.5 to
// 0.7 us less that way too). Blocks of 128 rows stage A half as often as blocks of
// 64, which pays where A's three planes are long: 4096 rows of 3072 columns, fp32 A
// of 64 ranks, 15.3 and 16.7 us. The rule goes by rows alone; with a bf16 A blocks
// of 64 rows are the faster ones (4096 x 12288 at rank 32 16.6 with blocks of 128 and
// 13.5 with blocks of 64, 128 rows 9.2 and 7.7). Target 512
// blocks, 256 and 1024 beside it: 2048 x 12288 13.2 us, 12.1, 13.2; 4096 16.6, 16.5, 17.0.
DownPlan down_plan(int64_t m, int64_t k, int64_t r) {
  DownPlan p;
  p.wr = m > 16 ? 4 : 1;
  p.fm = m > 64 ? 2 : 1;
  const int64_t rows = 16 * p.wr * p.fm;
  p.rb = (m + rows - 1) / rows;
  // (up to 24 splits: the join adds them eight at a time, and more only lengthen it)
  const int64_t want = p.rb > 0 ? 512 / p.rb : 0;
  split_of(m > 0 ? k / SD_KC : 0, want < 24 ? want : 24, &p.s, &p.cps);
  p.total = (int64_t)p.s * m * padded_rank(r);
  return p;
}

template <typename SRC, typename TB, int R>
hipError_t dt_launch(const SideGradArgs& a, const SidePlan& p, hipStream_t stream) {
  const DtArgs t{a.dy, a.lddy, a.b, a.ldb, a.m, a.n, a.r, p.s1, p.cps1, a.ws};
  const dim3 grid((unsigned)(p.rb * p.s1)), block(256);
  if (p.wr == 4)
    hipLaunchKernelGGL((k_side_dt<SRC, TB, R, 4>), grid, block, 0, stream, t);
  else
    hipLaunchKernelGGL((k_side_dt<SRC, TB, R, 1>), grid, block, 0, stream, t);
  return hipGetLastError();
}

template <int R>
hipError_t grad_r(const SideGradArgs& a, const SidePlan& p, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.m > 0) {
    if (a.n > 0) {
      if (a.dy_bf16)
        e = a.b_bf16 ? dt_launch<SrcBf16, uint16_t, R>(a, p, stream) : dt_launch<SrcBf16, float, R>(a, p, stream);
      else
        e = a.b_bf16 ? dt_launch<SrcF32, uint16_t, R>(a, p, stream) : dt_launch<SrcF32, float, R>(a, p, stream);
      if (e != hipSuccess) return e;
    }
    uint16_t *dt_planes = (uint16_t*)(a.ws + p.off4), *t_planes = (uint16_t*)(a.ws + p.off5);
    hipLaunchKernelGGL((k_side_prep<R>), dim3((unsigned)(2 * p.nmc)), dim3(512), 0, stream, a.ws, p.s1, a.m, a.sa,
                       a.alpha, a.r, a.t, a.dt, dt_planes, t_planes, p.nmc);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const OuterArgs db{a.dy, a.lddy, a.n, t_planes, a.m, p.s2, p.cps2, p.nmc, a.ws + p.off2};
    const OuterArgs da{a.qa, a.ldqa, a.k, dt_planes, a.m, p.s3, p.cps3, p.nmc, a.ws + p.off3};
    const unsigned nb_db = OuterShape<R>::blocks(p.cb2 * p.s2);
    const dim3 grid(nb_db + OuterShape<R>::blocks(p.cb3 * p.s3)), block(256);
    if (a.dy_bf16)
      hipLaunchKernelGGL((k_side_outer<SrcBf16, R>), grid, block, 0, stream, db, da, nb_db);
    else
      hipLaunchKernelGGL((k_side_outer<SrcF32, R>), grid, block, 0, stream, db, da, nb_db);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const unsigned nb_db = (unsigned)((a.n * (R / 4) + 1023) / 1024);
  const unsigned nb_da = (unsigned)(((int64_t)a.r * (a.k / 256) + 7) / 8);
  hipLaunchKernelGGL((k_side_join<R>), dim3(nb_db + nb_da), dim3(1024), 0, stream, a.ws + p.off2, p.s2, a.n, a.db,
                     a.lddb, a.alpha, a.ws + p.off3, p.s3, (int)a.k, a.da, a.ldda, a.rotate, a.r, nb_db);
  return hipGetLastError();
}

template <typename TA, int R>
hipError_t down_r(const SideDownArgs& a, hipStream_t stream) {
  const DownPlan p = down_plan(a.m, a.k, a.r);
  const DownArgs d{a.qa, a.ldqa, a.a, a.lda, a.m, a.r, p.s, p.cps, (int)(a.k / SD_KC), a.ws};
  const dim3 grid((unsigned)(p.rb * p.s)), block(256);
  if (p.wr == 1)
    hipLaunchKernelGGL((k_side_down<TA, R, 1, 1>), grid, block, 0, stream, d);
  else if (p.fm == 1)
    hipLaunchKernelGGL((k_side_down<TA, R, 4, 1>), grid, block, 0, stream, d);
  else
    hipLaunchKernelGGL((k_side_down<TA, R, 4, 2>), grid, block, 0, stream, d);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_side_join_t<R>), dim3((unsigned)((a.m * (SIDE_T / 4) + 255) / 256)), dim3(256), 0, stream, a.ws,
                     p.s, a.m, a.sa, a.r, a.t);
  return hipGetLastError();
}

template <typename TA>
hipError_t down_a(const SideDownArgs& a, hipStream_t stream) {
  if (a.r <= 16) return down_r<TA, 16>(a, stream);
  if (a.r <= 32) return down_r<TA, 32>(a, stream);
  return down_r<TA, 64>(a, stream);
}

}  // namespace

hipError_t launch_side_down(const SideDownArgs& a, hipStream_t stream) {
  return a.a_bf16 ? down_a<uint16_t>(a, stream) : down_a<float>(a, stream);
}

int64_t side_down_workspace_floats(int64_t m, int64_t k, int64_t r) { return down_plan(m, k, r).total; }

int64_t side_grad_workspace_floats(int64_t m, int64_t n, int64_t k, int64_t r) { return side_plan(m, n, k, r).total; }

hipError_t launch_side_grad(const SideGradArgs& a, hipStream_t stream) {
  const SidePlan p = side_plan(a.m, a.n, a.k, a.r);
  if (a.r <= 16) return grad_r<16>(a, p, stream);
  if (a.r <= 32) return grad_r<32>(a, p, stream);
  return grad_r<64>(a, p, stream);
}

}  // namespace tp
