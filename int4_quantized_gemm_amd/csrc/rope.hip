// Per-head RMS norm and rotary positions of q and k behind the qkv projection,
// and their gradients (the q/k norm and the rotary embedding among the row
// kernels around the projections, TensorFold pull request #948).
//
//   n  = x r gamma,  r = (mean(x^2) + eps)^(-1/2) per head (or n = x)
//   theta_p = position[axis(p)] f_p for the pairs p of a head
//   (a, b) -> (a cos theta - b sin theta, a sin theta + b cos theta)
//
// The angles of a token are the same for all its heads: a block takes a token
// at a time, works out the cosines and sines of its pairs once, into LDS, and
// turns every head of q and k with them. The angle is an fp64 product (a far
// position times a frequency does not fit in fp32), reduced to a fraction of a
// turn there and only then taken to fp32.
//
// Work layout: a lane holds four pairs of a head (8 elements: for interleaved
// pairs one run of 8, for halves a run of 4 in each half), a head takes
// head_dim / 8 lanes of a group of 2^g. Elements past the rotated pairs are
// taken as pairs that do not turn. Bound by HBM at many tokens.
#include "block_ops.hpp"
#include "device_common.hpp"

namespace tp {

constexpr int ROPE_THREADS = 256;
constexpr double TURN_HI = 0x1.45f306dc9c883p-3, TURN_LO = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)

__device__ __forceinline__ void load4(const void* p, int bf16, int64_t i, float (&v)[4]) {
  if (bf16) {
    const uint2 w = *reinterpret_cast<const uint2*>((const uint16_t*)p + i);
    v[0] = bf16_lo(w.x);
    v[1] = bf16_hi(w.x);
    v[2] = bf16_lo(w.y);
    v[3] = bf16_hi(w.y);
  } else {
    const f32x4_t w = *reinterpret_cast<const f32x4_t*>((const float*)p + i);
    v[0] = w.x;
    v[1] = w.y;
    v[2] = w.z;
    v[3] = w.w;
  }
}

__device__ __forceinline__ void store4(void* p, int bf16, int64_t i, const float (&v)[4]) {
  if (bf16)
    *reinterpret_cast<uint2*>((uint16_t*)p + i) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  else
    *reinterpret_cast<f32x4_t*>((float*)p + i) = f32x4_t{v[0], v[1], v[2], v[3]};
}

// Four pairs of a lane: a the first members, b the second ones.
struct Pairs {
  float a[4], b[4];
};

// Where a lane's pairs are in a head. Halves: pairs p are (p, P + p), then the
// rest of the head in halves of its own; interleaved: (2 p, 2 p + 1).
struct Where {
  int o0, o1;   // offsets of the lane's two runs of four elements
  int pair;     // its first pair; at or past the rotated ones: not turned
  bool on;      // the lane holds pairs at all
};

template <bool HALVES>
__device__ __forceinline__ Where where_of(int u, int d, int pairs) {
  Where w;
  w.on = 8 * u < d;
  w.pair = 4 * u;
  if (HALVES) {
    const int rest = (d - 2 * pairs) / 2;
    w.o0 = w.pair < pairs ? w.pair : 2 * pairs + (w.pair - pairs);
    w.o1 = w.o0 + (w.pair < pairs ? pairs : rest);
  } else {
    w.o0 = 8 * u;
    w.o1 = 8 * u + 4;
  }
  return w;
}

template <bool HALVES>
__device__ __forceinline__ void to_pairs(const float (&x)[4], const float (&y)[4], Pairs& p) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (HALVES) {
      p.a[e] = x[e];
      p.b[e] = y[e];
    } else {
      p.a[e] = e < 2 ? x[2 * e] : y[2 * e - 4];
      p.b[e] = e < 2 ? x[2 * e + 1] : y[2 * e - 3];
    }
  }
}

template <bool HALVES>
__device__ __forceinline__ void from_pairs(const Pairs& p, float (&x)[4], float (&y)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (HALVES) {
      x[e] = p.a[e];
      y[e] = p.b[e];
    } else if (e < 2) {
      x[2 * e] = p.a[e];
      x[2 * e + 1] = p.b[e];
    } else {
      y[2 * e - 4] = p.a[e];
      y[2 * e - 3] = p.b[e];
    }
  }
}

// Sum over the 2^g lanes that hold a head (the same tree in each of them).
__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int mask = 1; mask < lanes; mask <<= 1) v += __shfl_xor(v, mask);
  return v;
}

// The cosines and sines of a token's pairs. 1 / (2 pi) is taken in two doubles
// and the whole turns come off in one fma, so the fraction of a turn carries no
// more than the angle's own rounding; sincospif takes it from there.
__device__ __forceinline__ void token_turns(const RopeArgs& a, int64_t token, float2* turns) {
  for (int p = threadIdx.x; p < a.pairs; p += ROPE_THREADS) {
    const double angle = (double)a.positions[token * a.ldpos + a.axis[p]] * (double)a.inv_freq[p];
    const double turn = fma(angle, TURN_HI, -rint(angle * TURN_HI)) + angle * TURN_LO;
    float s, c;
    sincospif((float)(2.0 * turn), &s, &c);
    turns[p] = float2{c, s};
  }
}

// Forward (BWD false): out = R (x r gamma). Backward: g = R^T dy, then the
// norm's gradient where there is one, with dgamma kept per lane.
template <bool HALVES, bool BWD>
__global__ __launch_bounds__(ROPE_THREADS) void k_rope(RopeArgs a, int lanes, int units) {
  __shared__ float2 turns[2][ROPE_MAX_PAIRS];
  __shared__ float red[2][ROPE_THREADS][8];
  const int d = a.head_dim, heads = a.heads_q + a.heads_k;
  const int u = threadIdx.x & (lanes - 1), g0 = threadIdx.x / lanes, groups = ROPE_THREADS / lanes;
  const Where w = where_of<HALVES>(u, d, a.pairs);
  const float inv_d = 1.0f / (float)d, eps = fmaxf((float)a.eps, 0x1p-126f);
  // The block's slice of a token's heads, for few tokens (units slices).
  const int slice = (int)(blockIdx.x % (unsigned)units);
  const int h_begin = heads * slice / units, h_end = heads * (slice + 1) / units;
  const int64_t first = blockIdx.x / (unsigned)units, step = gridDim.x / (unsigned)units;

  Pairs gq, gk;  // weights
  {
    float x[4] = {1.f, 1.f, 1.f, 1.f}, y[4] = {1.f, 1.f, 1.f, 1.f};
    if (a.q_gamma.p && w.on) {
      load4(a.q_gamma.p, a.q_gamma.bf16, w.o0, x);
      load4(a.q_gamma.p, a.q_gamma.bf16, w.o1, y);
    }
    to_pairs<HALVES>(x, y, gq);
  }
  {
    float x[4] = {1.f, 1.f, 1.f, 1.f}, y[4] = {1.f, 1.f, 1.f, 1.f};
    if (a.k_gamma.p && w.on) {
      load4(a.k_gamma.p, a.k_gamma.bf16, w.o0, x);
      load4(a.k_gamma.p, a.k_gamma.bf16, w.o1, y);
    }
    to_pairs<HALVES>(x, y, gk);
  }
  Pairs sq, sk;  // dgamma of this lane's pairs
#pragma unroll
  for (int e = 0; e < 4; ++e) sq.a[e] = sq.b[e] = sk.a[e] = sk.b[e] = 0.f;

  int parity = 0;
  for (int64_t token = first; token < a.m; token += step, parity ^= 1) {
    token_turns(a, token, turns[parity]);
    __syncthreads();  // (slower threads may still read the other parity's turns)
    Pairs t;  // cosines and sines of the lane's pairs
    const bool turned = w.pair < a.pairs;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 cs = turned ? turns[parity][w.pair + e] : float2{1.f, 0.f};
      t.a[e] = cs.x;
      t.b[e] = BWD ? -cs.y : cs.y;
    }
    for (int hb = h_begin; hb < h_end; hb += groups) {  // the same count in every lane: they exchange
      const int h = hb + g0;
      const bool live = h < h_end && w.on;
      const bool is_q = h < a.heads_q;
      const int head = is_q ? h : h - a.heads_q;
      const bool norm = is_q ? a.q_gamma.p != nullptr : a.k_gamma.p != nullptr;
      const Pairs& gm = is_q ? gq : gk;
      const int64_t off = (int64_t)head * d;
      float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
      Pairs x, y;
      if (!BWD || norm) {
        if (live) {
          const void* src = is_q ? a.q : a.k;
          const int64_t i = token * (is_q ? a.ldq : a.ldk) + off;
          load4(src, a.x_bf16, i + w.o0, x0);
          load4(src, a.x_bf16, i + w.o1, x1);
        }
      }
      to_pairs<HALVES>(x0, x1, x);
      if (BWD) {
        float y0[4] = {0.f, 0.f, 0.f, 0.f}, y1[4] = {0.f, 0.f, 0.f, 0.f};
        if (live) {
          const void* src = is_q ? a.dq_out : a.dk_out;
          const int64_t i = token * (is_q ? a.lddqo : a.lddko) + off;
          load4(src, a.dy_bf16, i + w.o0, y0);
          load4(src, a.dy_bf16, i + w.o1, y1);
        }
        to_pairs<HALVES>(y0, y1, y);
      }
      float r = 1.f;
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(x.a[e], x.a[e], fmaf(x.b[e], x.b[e], ss));
        ss = group_sum(ss, lanes);
        r = 1.0f / sqrtf(fmaf(ss, inv_d, eps));
      }
      Pairs o;
      if (!BWD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float na = norm ? x.a[e] * r * gm.a[e] : x.a[e], nb = norm ? x.b[e] * r * gm.b[e] : x.b[e];
          o.a[e] = turned ? na * t.a[e] - nb * t.b[e] : na;
          o.b[e] = turned ? na * t.b[e] + nb * t.a[e] : nb;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o.a[e] = turned ? y.a[e] * t.a[e] - y.b[e] * t.b[e] : y.a[e];
          o.b[e] = turned ? y.a[e] * t.b[e] + y.b[e] * t.a[e] : y.b[e];
        }
        if (norm) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s = fmaf(o.a[e] * gm.a[e], x.a[e], fmaf(o.b[e] * gm.b[e], x.b[e], s));
          s = group_sum(s, lanes);
          const float coef = s * inv_d * r * r * r;
          Pairs& sg = is_q ? sq : sk;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sg.a[e] = fmaf(o.a[e] * r, x.a[e], sg.a[e]);
            sg.b[e] = fmaf(o.b[e] * r, x.b[e], sg.b[e]);
            o.a[e] = fmaf(o.a[e] * gm.a[e], r, -x.a[e] * coef);
            o.b[e] = fmaf(o.b[e] * gm.b[e], r, -x.b[e] * coef);
          }
        }
      }
      if (live) {
        float o0[4], o1[4];
        from_pairs<HALVES>(o, o0, o1);
        void* dst = is_q ? a.q_out : a.k_out;
        const int64_t i = token * (is_q ? a.ldqo : a.ldko) + off;
        store4(dst, a.out_bf16, i + w.o0, o0);
        store4(dst, a.out_bf16, i + w.o1, o1);
      }
    }
  }
  if (BWD && a.want_dgamma) {  // the block's dgamma: its groups added in order
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      red[0][threadIdx.x][e] = sq.a[e];
      red[0][threadIdx.x][4 + e] = sq.b[e];
      red[1][threadIdx.x][e] = sk.a[e];
      red[1][threadIdx.x][4 + e] = sk.b[e];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * d; e += ROPE_THREADS) {
      // element i of the head's weight: which lane and which of its 8 holds it
      const int i = e % d, qk = e / d;
      int lane, slot;
      if (HALVES) {
        const int rest = (d - 2 * a.pairs) / 2;
        const bool turned = i < 2 * a.pairs;
        const int j = turned ? i : i - 2 * a.pairs, half = turned ? a.pairs : rest;
        const int second = j >= half, p = (second ? j - half : j) + (turned ? 0 : a.pairs);
        lane = p >> 2;
        slot = 4 * second + (p & 3);
      } else {
        lane = i >> 3;
        slot = 4 * (i & 1) + ((i & 7) >> 1);
      }
      float s = 0.f;
      for (int g = 0; g < groups; ++g) s += red[qk][g * lanes + lane][slot];
      a.part[(int64_t)blockIdx.x * (2 * d) + e] = s;
    }
  }
}

namespace {

struct RopeShape {
  int lanes, units;
  int64_t blocks;
};

constexpr int64_t ROPE_BLOCKS = 8192, ROPE_BWD_BLOCKS = 1024;  // blocks walk tokens beyond that many

RopeShape rope_shape(int64_t m, int heads, int d, int64_t max_blocks) {
  RopeShape s;
  s.lanes = 1;
  while (s.lanes * 8 < d) s.lanes *= 2;
  const int groups = ROPE_THREADS / s.lanes;
  // few tokens: a token's heads go to several blocks
  int most = (heads + groups - 1) / groups;
  if (most < 1) most = 1;
  int64_t want = m > 0 ? 512 / m : 1;
  s.units = (int)(want < 1 ? 1 : want > most ? most : want);
  s.blocks = m * s.units;
  if (s.blocks > max_blocks) s.blocks = max_blocks / s.units * s.units;
  return s;
}

}  // namespace

int64_t rope_partial_rows(int64_t m, int heads, int d) {
  return rope_shape(m, heads, d, ROPE_BWD_BLOCKS).blocks;
}

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  const int heads = a.heads_q + a.heads_k;
  const RopeShape s = rope_shape(a.m, heads, a.head_dim, a.backward ? ROPE_BWD_BLOCKS : ROPE_BLOCKS);
  const dim3 grid((unsigned)s.blocks), block(ROPE_THREADS);
  if (s.blocks > 0) {
    if (a.backward) {
      if (a.halves)
        hipLaunchKernelGGL((k_rope<true, true>), grid, block, 0, stream, a, s.lanes, s.units);
      else
        hipLaunchKernelGGL((k_rope<false, true>), grid, block, 0, stream, a, s.lanes, s.units);
    } else {
      if (a.halves)
        hipLaunchKernelGGL((k_rope<true, false>), grid, block, 0, stream, a, s.lanes, s.units);
      else
        hipLaunchKernelGGL((k_rope<false, false>), grid, block, 0, stream, a, s.lanes, s.units);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.want_dgamma) return hipSuccess;
  return launch_colsum(a.part, s.blocks, 2 * (int64_t)a.head_dim, a.dq_gamma, a.head_dim, a.dk_gamma, stream);
}

}  // namespace tp
