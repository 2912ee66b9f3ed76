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

// --------------------------------------------------------------------- down
// A block owns 16 rows; its 16 waves share the K / 64 steps and add their
// sums in LDS in wave order. Lane l feeds row l % 16 with the 16 codes
// 16 (l / 16) of each step, and the same 16 columns of lora_a row l % 16.
constexpr int SD_WAVES = 16;

template <typename TA, int R>
__global__ __launch_bounds__(64 * SD_WAVES) void k_side_down(const int8_t* __restrict__ qa, int64_t ldqa,
                                                             const float* __restrict__ sa, const TA* __restrict__ a,
                                                             int64_t lda, int64_t M, int K, int r,
                                                             float* __restrict__ t) {
  constexpr int NF = R / 16;
  constexpr int PA = std::is_same<TA, float>::value ? 3 : 1;
  __shared__ __align__(16) float part[SD_WAVES][16][R];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int nk = K / 64, s0 = wave * nk / SD_WAVES, s1 = (wave + 1) * nk / SD_WAVES;
  const TA* arow[NF];
  int aval[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int j = f * 16 + l16;
    aval[f] = j < r ? 8 : 0;
    arow[f] = a + (int64_t)min(j, r - 1) * lda + 16 * g4;
  }
  for (int64_t m0 = (int64_t)blockIdx.x * 16; m0 < M; m0 += (int64_t)gridDim.x * 16) {
    const bool rowok = m0 + l16 < M;
    const int8_t* xrow = qa + min(m0 + l16, M - 1) * ldqa + 16 * g4;
    f32x4_t acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s = s0; s < s1; ++s) {
      u32x4_t w = {0u, 0u, 0u, 0u};
      if (rowok) w = *reinterpret_cast<const u32x4_t*>(xrow + 64 * s);
      const bf16x8_t x0[1] = {widen8(w.x, w.y)}, x1[1] = {widen8(w.z, w.w)};
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        bf16x8_t a0[PA], a1[PA];
        load_parts(arow[f] + 64 * s, aval[f], a0);
        load_parts(arow[f] + 64 * s + 8, aval[f], a1);
        acc[f] = mfma_parts(x0, a0, acc[f]);
        acc[f] = mfma_parts(x1, a1, acc[f]);
      }
    }
    // lane l holds rows 4 (l / 16) + v, column 16 f + l % 16
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][4 * g4 + v][f * 16 + l16] = acc[f][v];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * SIDE_T; e += 64 * SD_WAVES) {
      const int i = e / SIDE_T, j = e % SIDE_T;
      if (m0 + i >= M) continue;
      float sum = 0.f;
      if (j < R && j < r) {
        sum = part[0][i][j];
#pragma unroll
        for (int w = 1; w < SD_WAVES; ++w) sum += part[w][i][j];
        sum *= sa[m0 + i];
      }
      t[(m0 + i) * SIDE_T + j] = sum;
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------------- dt
// Partial sums of dY . B: a block owns 16 WR rows and a run of 256-column
// chunks; the chunk of B is transposed (and split) into LDS, from where it is
// the matrix units' second operand, and dY goes straight from memory to the
// first. With few rows (WR 1) the four waves share the chunk instead.
constexpr int DT_NC = 256;            // columns of dY per chunk
constexpr int DT_PITCH = DT_NC + 8;   // bf16 per LDS row: rows 4 banks apart

// Two dwords' low (odd == 0) or high halves in one.
__device__ __forceinline__ uint32_t pair_of(uint32_t first, uint32_t second, int odd) {
  return __builtin_amdgcn_perm(second, first, odd ? 0x07060302u : 0x05040100u);
}

// An 8 x 8 block of B (rows n, columns j) into the planes bt[part][j][n].
__device__ __forceinline__ void stage_b8(const uint16_t* b, int64_t ldb, int rows, int cols, uint16_t* bt, int,
                                         int pitch) {
  u32x4_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bf16x8_t o[1];
    load_parts(b + (int64_t)min(i, max(rows - 1, 0)) * ldb, i < rows ? cols : 0, o);
    w[i] = __builtin_bit_cast(u32x4_t, o[0]);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    u32x4_t o;
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = pair_of(w[2 * p][c >> 1], w[2 * p + 1][c >> 1], c & 1);
    *reinterpret_cast<u32x4_t*>(bt + c * pitch) = o;
  }
}

__device__ __forceinline__ void stage_b8(const float* b, int64_t ldb, int rows, int cols, uint16_t* bt, int plane,
                                         int pitch) {
  float w[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load_f32x8(b + (int64_t)min(i, max(rows - 1, 0)) * ldb, i < rows ? cols : 0, w[i]);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i][c];
    bf16x8_t h, m, l;
    split3_bf16(v, h, m, l);
    *reinterpret_cast<bf16x8_t*>(bt + c * pitch) = h;
    *reinterpret_cast<bf16x8_t*>(bt + plane + c * pitch) = m;
    *reinterpret_cast<bf16x8_t*>(bt + 2 * plane + c * pitch) = l;
  }
}

template <typename SRC, typename TB, int R, int WR>
__global__ __launch_bounds__(256) void k_side_dt(const typename SRC::elem* __restrict__ dy, int64_t lddy,
                                                 const TB* __restrict__ b, int64_t ldb, int64_t M, int64_t N, int r,
                                                 int splits, int chunks_per_split, float* __restrict__ part) {
  constexpr int NF = R / 16;
  constexpr int PY = SRC::PARTS, PB = std::is_same<TB, float>::value ? 3 : 1;
  constexpr int WN = 4 / WR;                // waves that share a chunk
  constexpr int STEPS = DT_NC / 32 / WN;    // 32-column steps of a wave and chunk
  constexpr int PLANE = R * DT_PITCH;
  __shared__ __align__(16) uint16_t bt[PB * PLANE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int rg = wave % WR, ns = wave / WR;
  const int split = (int)(blockIdx.x % (unsigned)splits);
  const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)splits) * (16 * WR) + 16 * rg;
  const bool rowok = m0 + l16 < M;
  const typename SRC::elem* row = dy + min(m0 + l16, M - 1) * lddy;
  const int64_t nchunks = (N + DT_NC - 1) / DT_NC;
  const int64_t c0 = (int64_t)split * chunks_per_split, c1 = min(c0 + chunks_per_split, nchunks);
  f32x4_t acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int64_t c = c0; c < c1; ++c) {
    const int64_t n0 = c * DT_NC;
    __syncthreads();
    for (int u = threadIdx.x; u < (DT_NC / 8) * (R / 8); u += 256) {
      const int nb = u / (R / 8), jb = u % (R / 8);
      const int64_t n = n0 + 8 * nb;
      const int rows = (int)max((int64_t)0, min((int64_t)8, N - n)), cols = max(0, min(8, r - 8 * jb));
      stage_b8(b + min(n, N - 1) * ldb + (cols > 0 ? 8 * jb : 0), ldb, rows, cols,
               bt + 8 * jb * DT_PITCH + 8 * nb, PLANE, DT_PITCH);
    }
    __syncthreads();
    const int64_t nw = n0 + ns * (32 * STEPS);
    bf16x8_t y[STEPS][PY];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int64_t n = nw + 32 * s + 8 * g4;
      const int valid = rowok ? (int)max((int64_t)0, min((int64_t)8, N - n)) : 0;
      load_parts(row + (valid > 0 ? n : 0), valid, y[s]);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        bf16x8_t bp[PB];
#pragma unroll
        for (int p = 0; p < PB; ++p)
          bp[p] = *reinterpret_cast<const bf16x8_t*>(bt + p * PLANE + (16 * f + l16) * DT_PITCH + ns * (32 * STEPS) +
                                                     32 * s + 8 * g4);
        acc[f] = mfma_parts(y[s], bp, acc[f]);
      }
  }
  float* out = part + ((int64_t)(split * WN + ns) * M + m0) * R;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (m0 + 4 * g4 + v < M) {
#pragma unroll
      for (int f = 0; f < NF; ++f) out[(int64_t)(4 * g4 + v) * R + 16 * f + l16] = acc[f][v];
    }
}

// -------------------------------------------------------------------- outer
// Partial sums over rows of small^T . big: small [rows, r] fp32 (T, or dT sa)
// split into three bf16 planes in LDS, big [rows, width] streamed from memory.
// The sum runs over the rows, so a lane loads an 8 x 8 block (8 rows, 8
// columns) and pairs up rows with byte permutes: its column c is then an
// operand of 8 consecutive rows, and 16 lanes cover 128 columns, every eighth
// at a time. A block's four waves own 128 columns each and a run of 64-row
// chunks.
constexpr int OU_MC = 64;            // rows per chunk
constexpr int OU_PITCH = OU_MC + 8;  // bf16 per LDS row
constexpr int OU_COLS = 512;         // columns of a block

template <typename SRC> struct Block8;  // 8 x 8 elements of a lane, and column c as an operand

template <> struct Block8<SrcBf16> {
  u32x4_t w[8];
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

template <> struct Block8<SrcF32> {
  float w[8][8];
  __device__ __forceinline__ void load(int i, const float* p, int valid) { load_f32x8(p, valid, w[i]); }
  __device__ __forceinline__ void column(int c, bf16x8_t (&o)[3]) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i][c];
    split3_bf16(v, o[0], o[1], o[2]);
  }
};

template <> struct Block8<SrcI8> {
  uint2 w[8];
  __device__ __forceinline__ void load(int i, const int8_t* p, int valid) {  // whole 8s: k is a multiple of 256
    w[i] = valid > 0 ? *reinterpret_cast<const uint2*>(p) : uint2{0u, 0u};
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

struct OuterArgs {
  const void* big;
  int64_t ldbig, width;   // [m, width]
  const float* small;     // T [m, 64] (dB), or the dt partial sums [np, m, R] (dA)
  int np;                 // partial sums to join; 0 with T
  float alpha;            // dA: factor of the joined sums
  const float* sa;        // dA: row scales
  float* dt;              // dA: dT [m, 64] to write
  int64_t m;
  int r, splits, chunks_per_split;
  int64_t nmc;            // 64-row chunks
  float* part;            // dB: [splits, width, R]; dA: [splits, R, width]
};

template <typename SRC, int R, bool DA>
__global__ __launch_bounds__(256) void k_side_outer(OuterArgs a) {
  constexpr int NF = R / 16, PS = SRC::PARTS;
  constexpr int PLANE = R * OU_PITCH;
  __shared__ __align__(16) uint16_t st[3 * PLANE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int split = (int)(blockIdx.x % (unsigned)a.splits);
  const int64_t cblk = blockIdx.x / (unsigned)a.splits;
  const int64_t col = cblk * OU_COLS + wave * 128 + 8 * l16;
  const int valid_cols = (int)max((int64_t)0, min((int64_t)8, a.width - col));
  const typename SRC::elem* big = (const typename SRC::elem*)a.big + (valid_cols > 0 ? col : 0);
  const int64_t c0 = (int64_t)split * a.chunks_per_split, c1 = min(c0 + a.chunks_per_split, a.nmc);
  f32x4_t acc[8][NF];
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[c][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int64_t ch = c0; ch < c1; ++ch) {
    const int64_t mb = ch * OU_MC;
    __syncthreads();
    for (int u = threadIdx.x; u < R * (OU_MC / 8); u += 256) {
      const int j = u % R, oct = u / R;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t row = mb + 8 * oct + i;
        v[i] = 0.f;
        if (row < a.m) {
          if constexpr (DA) {
            float s = 0.f;
            for (int p = 0; p < a.np; ++p) s += a.small[((int64_t)p * a.m + row) * R + j];
            s *= a.alpha;
            if (j >= a.r) s = 0.f;
            if (cblk == 0) a.dt[row * SIDE_T + j] = s;
            v[i] = s * a.sa[row];
          } else {
            if (j < a.r) v[i] = a.small[row * SIDE_T + j];
          }
        }
      }
      bf16x8_t h, md, l;
      split3_bf16(v, h, md, l);
      uint16_t* to = st + j * OU_PITCH + 8 * oct;
      *reinterpret_cast<bf16x8_t*>(to) = h;
      *reinterpret_cast<bf16x8_t*>(to + PLANE) = md;
      *reinterpret_cast<bf16x8_t*>(to + 2 * PLANE) = l;
    }
    if (DA && R < SIDE_T && cblk == 0) {  // dT is zero past the columns computed here
      constexpr int REST = SIDE_T - R;
      for (int u = threadIdx.x; u < OU_MC * REST; u += 256) {
        const int64_t row = mb + u / REST;
        if (row < a.m) a.dt[row * SIDE_T + R + u % REST] = 0.f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int sub = 0; sub < OU_MC / 32; ++sub) {
      Block8<SRC> blk;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t row = mb + 32 * sub + 8 * g4 + i;
        blk.load(i, big + min(row, a.m - 1) * a.ldbig, row < a.m ? valid_cols : 0);
      }
      bf16x8_t sm[NF][3];
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int p = 0; p < 3; ++p)
          sm[f][p] = *reinterpret_cast<const bf16x8_t*>(st + p * PLANE + (16 * f + l16) * OU_PITCH + 32 * sub + 8 * g4);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        bf16x8_t big_c[PS];
        blk.column(c, big_c);
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[c][f] = mfma_parts(sm[f], big_c, acc[c][f]);
      }
    }
  }
  // lane l holds, for column col + c, the ranks 16 f + 4 (l / 16) + v
  if constexpr (DA) {
    if (valid_cols > 0) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float o[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) o[c] = acc[c][f][v];
          store8(a.part + ((int64_t)split * R + 16 * f + 4 * g4 + v) * a.width + col, o);
        }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < valid_cols) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
          *reinterpret_cast<f32x4_t*>(a.part + ((int64_t)split * a.width + col + c) * R + 16 * f + 4 * g4) = acc[c][f];
      }
  }
}

// --------------------------------------------------------------------- join
// The splits of dB and dA added in order. The first nb_db blocks take dB, four
// ranks a thread; the others dA, a 256-group of one rank per half wave, which
// rotates it back on request.
template <int R>
__global__ __launch_bounds__(256) void k_side_join(const float* __restrict__ pb, int sb, int64_t N, float alpha,
                                                   float* __restrict__ db, int64_t lddb,
                                                   const float* __restrict__ pa, int sa_splits, int K,
                                                   float* __restrict__ da, int64_t ldda, int rotate, int r,
                                                   int64_t nb_db) {
  if ((int64_t)blockIdx.x < nb_db) {
    constexpr int Q = R / 4;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n = e / Q;
    const int j = (int)(e % Q) * 4;
    if (n >= N || j >= r) return;
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = 0; p < sb; ++p) s += *reinterpret_cast<const f32x4_t*>(pb + ((int64_t)p * N + n) * R + j);
    float* to = db + n * lddb + j;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (j + v < r) to[v] = s[v] * alpha;
    return;
  }
  const int lane32 = threadIdx.x & 31;
  const int groups = K / 256;
  const int64_t unit = ((int64_t)blockIdx.x - nb_db) * 8 + (threadIdx.x >> 5);
  if (unit >= (int64_t)r * groups) return;  // uniform over the half wave that owns the unit
  const int64_t j = unit / groups;
  const int64_t c = (unit % groups) * 256 + lane32 * 8;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
  for (int p = 0; p < sa_splits; ++p) {
    float w[8];
    load8(pa + ((int64_t)p * R + j) * K + c, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
  }
  if (rotate) {
    fwht256_lane8(v, lane32);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= 0.0625f;
  }
  store8(da + j * ldda + c, v);
}

// ---------------------------------------------------------------- launchers
namespace {

// How the sums are split: enough blocks for the chip, as few partial sums as
// that allows.
struct SidePlan {
  int R, wr;                     // padded rank; row groups of a dt block
  int64_t rb, nchunks;           // row blocks, 256-column chunks (dt)
  int s1, cps1, wn;              // splits of the columns, chunks of a split, partial sums per split
  int64_t nmc;                   // 64-row chunks (outer)
  int64_t cb2, cb3;              // column blocks of dB and dA
  int s2, cps2, s3, cps3;
  int64_t off2, off3, total;     // floats: the dB and dA partial sums, and all
};

void split_of(int64_t chunks, int64_t want, int* splits, int* per) {
  if (chunks == 0) {
    *splits = 0;
    *per = 0;
    return;
  }
  int64_t s = want < 1 ? 1 : (want > chunks ? chunks : want);
  const int64_t p = (chunks + s - 1) / s;
  *per = (int)p;
  *splits = (int)((chunks + p - 1) / p);
}

SidePlan side_plan(int64_t m, int64_t n, int64_t k, int64_t r) {
  SidePlan p;
  p.R = r <= 16 ? 16 : r <= 32 ? 32 : 64;
  p.wr = m > 16 ? 4 : 1;
  p.wn = 4 / p.wr;
  p.rb = (m + 16 * p.wr - 1) / (16 * p.wr);
  p.nchunks = (n + DT_NC - 1) / DT_NC;
  split_of(m > 0 ? p.nchunks : 0, p.rb > 0 ? 512 / p.rb : 0, &p.s1, &p.cps1);
  p.nmc = (m + OU_MC - 1) / OU_MC;
  p.cb2 = (n + OU_COLS - 1) / OU_COLS;
  p.cb3 = (k + OU_COLS - 1) / OU_COLS;
  split_of(n > 0 ? p.nmc : 0, p.cb2 > 0 ? 256 / p.cb2 : 0, &p.s2, &p.cps2);
  split_of(p.nmc, 256 / p.cb3 < 16 ? 256 / p.cb3 : 16, &p.s3, &p.cps3);
  p.off2 = (int64_t)p.s1 * p.wn * m * p.R;
  p.off3 = p.off2 + (int64_t)p.s2 * n * p.R;
  p.total = p.off3 + (int64_t)p.s3 * k * p.R;
  return p;
}

template <typename SRC, typename TB, int R>
hipError_t dt_launch(const SideGradArgs& a, const SidePlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)(p.rb * p.s1)), block(256);
  if (p.wr == 4)
    hipLaunchKernelGGL((k_side_dt<SRC, TB, R, 4>), grid, block, 0, stream, (const typename SRC::elem*)a.dy, a.lddy,
                       (const TB*)a.b, a.ldb, a.m, a.n, a.r, p.s1, p.cps1, a.ws);
  else
    hipLaunchKernelGGL((k_side_dt<SRC, TB, R, 1>), grid, block, 0, stream, (const typename SRC::elem*)a.dy, a.lddy,
                       (const TB*)a.b, a.ldb, a.m, a.n, a.r, p.s1, p.cps1, a.ws);
  return hipGetLastError();
}

template <int R>
hipError_t grad_r(const SideGradArgs& a, const SidePlan& p, hipStream_t stream) {
  hipError_t e = hipSuccess;
  const dim3 block(256);
  if (p.s1 > 0) {
    if (a.dy_bf16)
      e = a.b_bf16 ? dt_launch<SrcBf16, uint16_t, R>(a, p, stream) : dt_launch<SrcBf16, float, R>(a, p, stream);
    else
      e = a.b_bf16 ? dt_launch<SrcF32, uint16_t, R>(a, p, stream) : dt_launch<SrcF32, float, R>(a, p, stream);
    if (e != hipSuccess) return e;
  }
  OuterArgs o{};
  o.m = a.m;
  o.r = a.r;
  o.nmc = p.nmc;
  if (p.s2 > 0) {
    o.big = a.dy;
    o.ldbig = a.lddy;
    o.width = a.n;
    o.small = a.t;
    o.splits = p.s2;
    o.chunks_per_split = p.cps2;
    o.part = a.ws + p.off2;
    const dim3 grid((unsigned)(p.cb2 * p.s2));
    if (a.dy_bf16)
      hipLaunchKernelGGL((k_side_outer<SrcBf16, R, false>), grid, block, 0, stream, o);
    else
      hipLaunchKernelGGL((k_side_outer<SrcF32, R, false>), grid, block, 0, stream, o);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (p.s3 > 0) {
    o.big = a.qa;
    o.ldbig = a.ldqa;
    o.width = a.k;
    o.small = a.ws;
    o.np = p.s1 * p.wn;
    o.alpha = a.alpha;
    o.sa = a.sa;
    o.dt = a.dt;
    o.splits = p.s3;
    o.chunks_per_split = p.cps3;
    o.part = a.ws + p.off3;
    hipLaunchKernelGGL((k_side_outer<SrcI8, R, true>), dim3((unsigned)(p.cb3 * p.s3)), block, 0, stream, o);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const int64_t nb_db = (a.n * (R / 4) + 255) / 256;
  const int64_t nb_da = ((int64_t)a.r * (a.k / 256) + 7) / 8;
  hipLaunchKernelGGL((k_side_join<R>), dim3((unsigned)(nb_db + nb_da)), block, 0, stream, a.ws + p.off2, p.s2, a.n,
                     a.alpha, a.db, a.lddb, a.ws + p.off3, p.s3, (int)a.k, a.da, a.ldda, a.rotate, a.r, nb_db);
  return hipGetLastError();
}

template <typename TA>
hipError_t down_a(const int8_t* qa, int64_t ldqa, const float* sa, const TA* a, int64_t lda, int64_t m, int64_t k,
                  int r, float* t, hipStream_t stream) {
  const int64_t rb = (m + 15) / 16;
  const dim3 grid((unsigned)(rb < 65536 ? rb : 65536)), block(64 * SD_WAVES);
#define TP_SIDE_DOWN(R) \
  hipLaunchKernelGGL((k_side_down<TA, R>), grid, block, 0, stream, qa, ldqa, sa, a, lda, m, (int)k, r, t)
  if (r <= 16)
    TP_SIDE_DOWN(16);
  else if (r <= 32)
    TP_SIDE_DOWN(32);
  else
    TP_SIDE_DOWN(64);
#undef TP_SIDE_DOWN
  return hipGetLastError();
}

}  // namespace

hipError_t launch_side_down(const int8_t* qa, int64_t ldqa, const float* sa, const void* a, bool a_bf16, int64_t lda,
                            int64_t m, int64_t k, int r, float* t, hipStream_t stream) {
  return a_bf16 ? down_a(qa, ldqa, sa, (const uint16_t*)a, lda, m, k, r, t, stream)
                : down_a(qa, ldqa, sa, (const float*)a, lda, m, k, r, t, stream);
}

int64_t side_grad_workspace_floats(int64_t m, int64_t n, int64_t k, int64_t r) { return side_plan(m, n, k, r).total; }

hipError_t launch_side_grad(const SideGradArgs& a, hipStream_t stream) {
  const SidePlan p = side_plan(a.m, a.n, a.k, a.r);
  if (p.R == 16) return grad_r<16>(a, p, stream);
  if (p.R == 32) return grad_r<32>(a, p, stream);
  return grad_r<64>(a, p, stream);
}

}  // namespace tp
