// Per-head RMS norm and rotary positions of q and k behind the qkv projection,
// and their gradients (the q/k norm and the rotary embedding among the row
// kernels around the projections, TensorFold pull request #948).
//
//   n  = x r gamma,  r = (mean(x^2) + eps)^(-1/2) per head (or n = x)
//   theta_p = position[axis(p)] f_p for the pairs p of a head
//   (a, b) -> (a cos theta - b sin theta, a sin theta + b cos theta)
//
// The angles of a token are the same for all its heads: a block takes a few
// tokens at a time, works out the cosines and sines of their pairs once, into
// LDS, and turns every head of q and k with them. The angle is an fp64 product (a far
// position times a frequency does not fit in fp32), reduced to a fraction of a
// turn there and only then taken to fp32.
//
// Work layout: a lane holds four pairs of a head (8 elements: for interleaved
// pairs one run of 8, for halves a run of 4 in each half), a head takes
// head_dim / 8 lanes of a group of 2^g. Elements past the rotated pairs are
// taken as pairs that do not turn. Bound by HBM at many tokens (4096 tokens of 48
// heads of 128: fp32 to bf16 29.4 us, 5.1 TB/s; gradients in bf16 34.7 us, 4.4
// TB/s, and 4.3 us for the join of the weights' partial sums).
#include "block_ops.hpp"
#include "device_common.hpp"

namespace tp {

constexpr int ROPE_THREADS = 256;
constexpr double TURN_HI = 0x1.45f306dc9c883p-3, TURN_LO = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)

// A lane's eight elements of a head: two runs of four.
template <typename T>
struct Eight;

template <>
struct Eight<uint16_t> {
  uint2 w[2];
  __device__ __forceinline__ void load(const uint16_t* p, int o0, int o1) {
    w[0] = *reinterpret_cast<const uint2*>(p + o0);
    w[1] = *reinterpret_cast<const uint2*>(p + o1);
  }
  __device__ __forceinline__ void load(const uint16_t* p) {  // one run of eight
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
    w[0] = uint2{v.x, v.y};
    w[1] = uint2{v.z, v.w};
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = uint2{0u, 0u}; }
  __device__ __forceinline__ void get(float (&x)[4], float (&y)[4]) const {
    x[0] = bf16_lo(w[0].x);
    x[1] = bf16_hi(w[0].x);
    x[2] = bf16_lo(w[0].y);
    x[3] = bf16_hi(w[0].y);
    y[0] = bf16_lo(w[1].x);
    y[1] = bf16_hi(w[1].x);
    y[2] = bf16_lo(w[1].y);
    y[3] = bf16_hi(w[1].y);
  }
  static __device__ __forceinline__ void store(uint16_t* p, int o0, int o1, const float (&x)[4], const float (&y)[4]) {
    *reinterpret_cast<uint2*>(p + o0) = uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    *reinterpret_cast<uint2*>(p + o1) = uint2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&x)[4], const float (&y)[4]) {
    *reinterpret_cast<u32x4_t*>(p) = u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                             pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
  }
};

template <>
struct Eight<float> {
  f32x4_t w[2];
  __device__ __forceinline__ void load(const float* p, int o0, int o1) {
    w[0] = *reinterpret_cast<const f32x4_t*>(p + o0);
    w[1] = *reinterpret_cast<const f32x4_t*>(p + o1);
  }
  __device__ __forceinline__ void load(const float* p) { load(p, 0, 4); }
  __device__ __forceinline__ void zero() { w[0] = w[1] = f32x4_t{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void get(float (&x)[4], float (&y)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = w[0][e];
      y[e] = w[1][e];
    }
  }
  static __device__ __forceinline__ void store(float* p, int o0, int o1, const float (&x)[4], const float (&y)[4]) {
    *reinterpret_cast<f32x4_t*>(p + o0) = f32x4_t{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4_t*>(p + o1) = f32x4_t{y[0], y[1], y[2], y[3]};
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[4], const float (&y)[4]) {
    store(p, 0, 4, x, y);
  }
};

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

// The cosines and sines of a token's pair. 1 / (2 pi) is taken in two doubles
// and the whole turns come off in one fma, so the fraction of a turn carries no
// more than the angle's own rounding; sincospif takes it from there.
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, int64_t token, int p) {
  const double angle = (double)a.positions[token * a.ldpos + a.axis[p]] * (double)a.inv_freq[p];
  const double turn = fma(angle, TURN_HI, -rint(angle * TURN_HI)) + angle * TURN_LO;
  float s, c;
  sincospif((float)(2.0 * turn), &s, &c);
  return float2{c, s};
}

// What the kernel needs of q or of k.
struct Heads {
  const void *x, *dy;
  void* out;
  int64_t ldx, lddy, ldout;
  VecArg gamma;
  int begin, count;  // the block's heads
};

// Forward (BWD false): out = R (x r gamma). Backward: g = R^T dy, then the
// norm's gradient where there is one, with dgamma kept per lane. A block takes
// `batch` tokens at a time (as many as its threads have pairs for) and a slice
// of their heads; the next head's elements are in flight while one is turned.
template <bool HALVES, bool BWD, typename TX, typename TY, typename TO>
__global__ __launch_bounds__(ROPE_THREADS) void k_rope(RopeArgs a, int lanes, int slices, int batch) {
  __shared__ __align__(16) float2 turns[ROPE_THREADS];
  __shared__ float red[2][ROPE_THREADS][8];
  const int d = a.head_dim;
  const int u = threadIdx.x & (lanes - 1), g0 = threadIdx.x / lanes, groups = ROPE_THREADS / lanes;
  const Where w = where_of<HALVES>(u, d, a.pairs);
  const bool turned = w.pair < a.pairs;
  const float inv_d = 1.0f / (float)d, eps = (float)a.eps;
  const int slice = (int)(blockIdx.x % (unsigned)slices);
  const int64_t first = (int64_t)(blockIdx.x / (unsigned)slices) * batch;
  const int64_t step = (int64_t)(gridDim.x / (unsigned)slices) * batch;

  auto weight = [&](const VecArg& g, Pairs& p) {
    float x[4] = {1.f, 1.f, 1.f, 1.f}, y[4] = {1.f, 1.f, 1.f, 1.f};
    if (g.p != nullptr && w.on) {
      if (g.bf16) {
        Eight<uint16_t> r;
        r.load((const uint16_t*)g.p, w.o0, w.o1);
        r.get(x, y);
      } else {
        Eight<float> r;
        r.load((const float*)g.p, w.o0, w.o1);
        r.get(x, y);
      }
    }
    to_pairs<HALVES>(x, y, p);
  };

  // One tensor's heads of the tokens t0 .. t0 + nt.
  auto run = [&](const Heads& h, const Pairs& gm, Pairs& sg, int64_t t0, int nt) {
    const bool norm = h.gamma.p != nullptr;
    const int total = nt * h.count;
    if (total == 0) return;
    Eight<TX> rx;
    Eight<TY> ry;
    auto fetch = [&](int64_t token, int head) {
      if (!BWD || norm) {
        const TX* p = (const TX*)h.x + token * h.ldx + (int64_t)head * d;
        if (HALVES) rx.load(p, w.o0, w.o1); else rx.load(p + w.o0);
      }
      if (BWD) {
        const TY* p = (const TY*)h.dy + token * h.lddy + (int64_t)head * d;
        if (HALVES) ry.load(p, w.o0, w.o1); else ry.load(p + w.o0);
      }
    };
    // (token, head) units, one a group of lanes; (t, c) walks them
    int t = g0 / h.count, c = g0 - t * h.count;
    rx.zero();
    if (BWD) ry.zero();
    if (w.on && t < nt) fetch(t0 + t, h.begin + c);
    for (int ub = 0; ub < total; ub += groups) {  // the same count in every lane: they exchange
      const bool live = w.on && t < nt;
      float x0[4], x1[4], y0[4], y1[4];
      rx.get(x0, x1);
      if (BWD) ry.get(y0, y1);
      const int64_t token = t0 + t;
      const int head = h.begin + c, tl = min(t, nt - 1);
      c += groups;
      while (c >= h.count) {
        c -= h.count;
        ++t;
      }
      if (w.on && t < nt) fetch(t0 + t, h.begin + c);
      Pairs x, cs;
      to_pairs<HALVES>(x0, x1, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = turned ? turns[tl * a.pairs + w.pair + e] : float2{1.f, 0.f};
        cs.a[e] = v.x;
        cs.b[e] = BWD ? -v.y : v.y;
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
          o.a[e] = turned ? na * cs.a[e] - nb * cs.b[e] : na;
          o.b[e] = turned ? na * cs.b[e] + nb * cs.a[e] : nb;
        }
      } else {
        Pairs y;
        to_pairs<HALVES>(y0, y1, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o.a[e] = turned ? y.a[e] * cs.a[e] - y.b[e] * cs.b[e] : y.a[e];
          o.b[e] = turned ? y.a[e] * cs.b[e] + y.b[e] * cs.a[e] : y.b[e];
        }
        if (norm) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) s = fmaf(o.a[e] * gm.a[e], x.a[e], fmaf(o.b[e] * gm.b[e], x.b[e], s));
          s = group_sum(s, lanes);
          // n = x r and r mean(gamma g x) are of the gradients' size; r^3 alone leaves
          // fp32 where the head's squares still fit
          const float mean = s * inv_d * r, rl = live ? r : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float na = x.a[e] * rl, nb = x.b[e] * rl;
            sg.a[e] = fmaf(o.a[e], na, sg.a[e]);
            sg.b[e] = fmaf(o.b[e], nb, sg.b[e]);
            o.a[e] = fmaf(-na, mean, o.a[e] * gm.a[e]) * r;
            o.b[e] = fmaf(-nb, mean, o.b[e] * gm.b[e]) * r;
          }
        }
      }
      if (live) {
        float o0[4], o1[4];
        from_pairs<HALVES>(o, o0, o1);
        TO* p = (TO*)h.out + token * h.ldout + (int64_t)head * d;
        if (HALVES) Eight<TO>::store(p, w.o0, w.o1, o0, o1); else Eight<TO>::store(p + w.o0, o0, o1);
      }
    }
  };

  auto slice_of = [&](int heads, int& begin, int& count) {
    begin = heads * slice / slices;
    count = heads * (slice + 1) / slices - begin;
  };
  Heads hq{a.q, a.dq_out, a.q_out, a.ldq, a.lddqo, a.ldqo, a.q_gamma, 0, 0};
  Heads hk{a.k, a.dk_out, a.k_out, a.ldk, a.lddko, a.ldko, a.k_gamma, 0, 0};
  slice_of(a.heads_q, hq.begin, hq.count);
  slice_of(a.heads_k, hk.begin, hk.count);
  Pairs gq, gk, sq, sk;  // weights, and this lane's part of their gradients
  weight(a.q_gamma, gq);
  weight(a.k_gamma, gk);
#pragma unroll
  for (int e = 0; e < 4; ++e) sq.a[e] = sq.b[e] = sk.a[e] = sk.b[e] = 0.f;

  for (int64_t t0 = first; t0 < a.m; t0 += step) {
    const int nt = (int)min((int64_t)batch, a.m - t0);
    __syncthreads();
    for (int e = threadIdx.x; e < nt * a.pairs; e += ROPE_THREADS)
      turns[e] = turn_of(a, t0 + e / a.pairs, e % a.pairs);
    __syncthreads();
    run(hq, gq, sq, t0, nt);
    run(hk, gk, sk, t0, nt);
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
        const bool first_part = i < 2 * a.pairs;
        const int j = first_part ? i : i - 2 * a.pairs, half = first_part ? a.pairs : rest;
        const int second = j >= half, p = (second ? j - half : j) + (first_part ? 0 : a.pairs);
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
  int lanes, slices, batch;
  int64_t blocks;
};

// Blocks walk tokens beyond that many. The gradients' blocks each write a partial
// row: 4096 tokens of 48 heads of 128 in bf16 41.1 us with 1024 blocks, 49.1 with 512,
// 41.1 with 2048; 16384 tokens 126.6, 166.0, 134.4.
constexpr int64_t ROPE_BLOCKS = 8192, ROPE_BWD_BLOCKS = 1024;

RopeShape rope_shape(int64_t m, int heads, int d, int pairs, int64_t max_blocks) {
  RopeShape s;
  s.lanes = 1;
  while (s.lanes * 8 < d) s.lanes *= 2;
  const int groups = ROPE_THREADS / s.lanes;
  // As many tokens at a time as the block's threads work out the turns of (4 at
  // most), but 1024 blocks, four a compute unit; with few tokens a token's heads go
  // to several blocks, 512 in all. Tokens of 48 heads of 128 in bf16, microseconds:
  //   at most 4 tokens, 2      4096: 25.8, 29.1      16384: 85.8, 81.2
  //   1024 blocks, 512, 2048   2048: 13.7, 16.7, 16.3      4096: 25.8, 25.7, 29.2
  //   512 slices, 256, 1024    256: 5.6, 6.9, 6.0      515: 8.5, 8.4, 8.5
  s.batch = pairs > 0 ? ROPE_THREADS / pairs : 4;
  if (s.batch > 4) s.batch = 4;
  while (s.batch > 1 && (m + s.batch - 1) / s.batch < 1024) s.batch /= 2;
  int most = (heads + groups - 1) / groups;
  if (most < 1) most = 1;
  const int64_t batches = (m + s.batch - 1) / s.batch;
  const int64_t want = batches > 0 ? 512 / batches : 1;
  s.slices = (int)(want < 1 ? 1 : want > most ? most : want);
  s.blocks = batches * s.slices;
  if (s.blocks > max_blocks) s.blocks = max_blocks / s.slices * s.slices;
  return s;
}

template <bool HALVES, typename TX, typename TO>
void rope_forward(const RopeArgs& a, const RopeShape& s, hipStream_t stream) {
  hipLaunchKernelGGL((k_rope<HALVES, false, TX, TX, TO>), dim3((unsigned)s.blocks), dim3(ROPE_THREADS), 0, stream, a,
                     s.lanes, s.slices, s.batch);
}

template <bool HALVES, typename TX, typename TY>
void rope_backward(const RopeArgs& a, const RopeShape& s, hipStream_t stream) {
  if (a.out_bf16)
    hipLaunchKernelGGL((k_rope<HALVES, true, TX, TY, uint16_t>), dim3((unsigned)s.blocks), dim3(ROPE_THREADS), 0,
                       stream, a, s.lanes, s.slices, s.batch);
  else
    hipLaunchKernelGGL((k_rope<HALVES, true, TX, TY, float>), dim3((unsigned)s.blocks), dim3(ROPE_THREADS), 0, stream,
                       a, s.lanes, s.slices, s.batch);
}

template <bool HALVES, typename TX>
void rope_x(const RopeArgs& a, const RopeShape& s, hipStream_t stream) {
  if (a.backward)
    a.dy_bf16 ? rope_backward<HALVES, TX, uint16_t>(a, s, stream) : rope_backward<HALVES, TX, float>(a, s, stream);
  else
    a.out_bf16 ? rope_forward<HALVES, TX, uint16_t>(a, s, stream) : rope_forward<HALVES, TX, float>(a, s, stream);
}

}  // namespace

int64_t rope_partial_rows(int64_t m, int heads, int d) {
  // (the most that any number of pairs asks for: the shape's batch goes by them)
  int64_t most = 0;
  for (int pairs = 0; pairs <= d / 2; pairs += 4) {
    const int64_t b = rope_shape(m, heads, d, pairs, ROPE_BWD_BLOCKS).blocks;
    most = b > most ? b : most;
  }
  return most;
}

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  const RopeShape s = rope_shape(a.m, a.heads_q + a.heads_k, a.head_dim, a.pairs,
                                 a.backward ? ROPE_BWD_BLOCKS : ROPE_BLOCKS);
  if (s.blocks > 0) {
    if (a.halves)
      a.x_bf16 ? rope_x<true, uint16_t>(a, s, stream) : rope_x<true, float>(a, s, stream);
    else
      a.x_bf16 ? rope_x<false, uint16_t>(a, s, stream) : rope_x<false, float>(a, s, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.want_dgamma) return hipSuccess;
  return launch_colsum(a.part, s.blocks, 2 * (int64_t)a.head_dim, a.dq_gamma, a.head_dim, a.dk_gamma, stream);
}

}  // namespace tp
