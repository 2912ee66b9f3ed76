// Internal launchers of the operators around the projections of a transformer
// block: norm.hip (RMS norm in front of them), side.hip (the adapter's side
// path on 8-bit activations, and its gradients) and rope.hip (per-head norm and
// rotary positions behind the qkv projection). Callers (api.cpp) validate every
// argument first; the launchers return the launch's hipError_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tp {

// A vector of weights: fp32 or bf16, or none (p == nullptr).
struct VecArg {
  const void* p;
  int bf16;
};

// ------------------------------------------------------------------ norm.hip
constexpr int NORM_MAX_GROUPS = 64;  // one 16-lane set per 256-group, 1024 threads a row at most

struct NormArgs {
  const void* x;
  int x_bf16;
  int64_t ldx;
  const void* res;  // nullptr: no residual (and no sum)
  int64_t ldr;
  void* sum;
  int64_t ldsum;
  int s_bf16;
  VecArg gamma;
  double eps;
  int rotate;
  int64_t m;
  int groups;
  int out_i8;
  void* y;
  int64_t ldy;
  float* scales;
};
hipError_t launch_norm_rotate(const NormArgs& a, hipStream_t stream);

struct NormBwdArgs {
  const void* dy;
  int dy_bf16;
  int64_t lddy;
  int rotate;
  const void* t;
  int t_bf16;
  int64_t ldt;
  VecArg gamma;
  double eps;
  const void* dsum;  // nullptr: none
  int64_t ldds;
  int64_t m;
  int groups;
  void* dx;
  int dx_bf16;
  int64_t lddx;
  float* dgamma;  // nullptr: not wanted
  float* part;    // norm_bwd_partial_rows(m, groups) rows of groups * 256 floats
};
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t stream);
int64_t norm_bwd_partial_rows(int64_t m, int groups);

// Sums over the rows of part [rows, cols], added in a fixed order: the first
// `first` columns to out, the others to out2 (null: not wanted).
hipError_t launch_colsum(const float* part, int64_t rows, int64_t cols, float* out, int64_t first, float* out2,
                         hipStream_t stream);

// ------------------------------------------------------------------ side.hip
struct SideDownArgs {  // T = sa (qa . a^T)
  const int8_t* qa;    // [m, k]
  int64_t ldqa;
  const float* sa;
  const void* a;  // [r, k]
  int a_bf16;
  int64_t lda, m, k;
  int r;
  float* t;   // [m, 64] (zeros past r)
  float* ws;  // side_down_workspace_floats(m, k, r) floats
};
hipError_t launch_side_down(const SideDownArgs& a, hipStream_t stream);
int64_t side_down_workspace_floats(int64_t m, int64_t k, int64_t r);

struct SideGradArgs {
  const void* dy;  // [m, n]
  int dy_bf16;
  int64_t lddy;
  const int8_t* qa;  // [m, k]
  int64_t ldqa;
  const float* sa;
  const float* t;  // [m, 64]
  const void* b;   // [n, r]
  int b_bf16;
  int64_t ldb;
  float alpha;
  int rotate;
  int64_t m, n, k;
  int r;
  float* dt;  // [m, 64]
  float* da;  // [r, k]
  int64_t ldda;
  float* db;  // [n, r]
  int64_t lddb;
  float* ws;  // side_grad_workspace_floats(m, n, k, r) floats
};
hipError_t launch_side_grad(const SideGradArgs& a, hipStream_t stream);
int64_t side_grad_workspace_floats(int64_t m, int64_t n, int64_t k, int64_t r);

// ------------------------------------------------------------------ rope.hip
constexpr int ROPE_MAX_DIM = 256, ROPE_MAX_PAIRS = ROPE_MAX_DIM / 2, ROPE_MAX_HEADS = 4096;

struct RopeArgs {
  const void *q, *k;  // [m, heads * head_dim]; the backward's only where there is a norm
  int64_t ldq, ldk;
  int x_bf16;
  int64_t m;
  int heads_q, heads_k, head_dim;
  VecArg q_gamma, k_gamma;  // none: no norm
  double eps;
  const int32_t* positions;  // [m, axes]
  int64_t ldpos;
  const float* inv_freq;  // [pairs]
  int pairs, halves;
  void *q_out, *k_out;  // the rotated heads, or their inputs' gradients
  int64_t ldqo, ldko;
  int out_bf16;
  int backward;
  const void *dq_out, *dk_out;
  int64_t lddqo, lddko;
  int dy_bf16;
  float *dq_gamma, *dk_gamma;  // null: not wanted
  int want_dgamma;             // either of them is
  float* part;                 // rope_partial_rows() rows of 2 head_dim floats, where want_dgamma
  uint8_t axis[ROPE_MAX_PAIRS];
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);
int64_t rope_partial_rows(int64_t m, int heads, int d);

// ----------------------------------------------------------------- philox.hpp
// A dropout: rng points at two 64-bit numbers in device memory, the seed and
// the offset (nullptr: none); threshold 0 .. 65536 of 16 random bits; scale
// 65536 / (65536 - threshold), 0 where everything drops.
struct DropArg {
  const uint64_t* rng;
  uint32_t threshold;
  float scale;
};

// -------------------------------------------------------------- layernorm.hip
struct LayerNormArgs {
  const void* x;
  int x_bf16;
  int64_t ldx;
  const void* res;  // nullptr: no residual (and no sum, and no dropout)
  int64_t ldr;
  void* sum;
  int64_t ldsum;
  int s_bf16;
  VecArg gamma, beta;
  double eps;
  DropArg drop;
  int rotate;
  int64_t m;
  int groups;
  int out;  // TP_NORM_OUT_*
  void* y;
  int64_t ldy;
  float* scales;
  int64_t ldscales;  // TP_NORM_OUT_FP8: [k / 128, m]
};
hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t stream);

struct LayerNormBwdArgs {
  const void* dy;
  int dy_bf16;
  int64_t lddy;
  int rotate;
  const void* t;
  int t_bf16;
  int64_t ldt;
  VecArg gamma;
  double eps;
  const void* dsum;  // nullptr: none
  int64_t ldds;
  DropArg drop;
  int64_t m;
  int groups;
  void* dx;
  int dx_bf16;
  int64_t lddx;
  void* dbranch;  // nullptr: not wanted (without drop.rng nothing drops: dx's values)
  int64_t lddb;
  float *dgamma, *dbeta;  // nullptr: not wanted
  float* part;            // layernorm_bwd_workspace_bytes(m, groups) bytes, where one is
  double* stats;          // (set by the launcher)
};
hipError_t launch_layernorm_bwd(const LayerNormBwdArgs& a, hipStream_t stream);
int64_t layernorm_bwd_workspace_bytes(int64_t m, int groups);

// ---------------------------------------------------------------- dropout.hip
struct DropoutArgs {
  const void* x;  // [m, k]
  int x_bf16;
  int64_t ldx;
  const void* res;  // nullptr: none; of y's type
  int64_t ldr;
  DropArg drop;
  int64_t m, k;
  void* y;
  int y_bf16;
  int64_t ldy;
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t stream);

// -------------------------------------------------------------------- fp8.hip
struct QuantFp8Args {
  const void* x;  // [m, k]
  int x_bf16;
  int64_t ldx;
  int64_t m, k;
  int rotate;   // k a multiple of 256
  int blocks;   // a scale per 128 x 128 block (else per 128 elements of a row, or of a column)
  uint8_t* q;   // [m, kp] codes, kp = k rounded up to 128 (nullptr: not wanted)
  int64_t ldq;
  float* s;     // [kp / 128, m], or with blocks [mp / 128, kp / 128]
  int64_t lds;
  uint8_t* qt;  // [k, mp] codes of the transpose (nullptr: not wanted)
  int64_t ldqt;
  float* st;    // [mp / 128, k], or with blocks [kp / 128, mp / 128]
  int64_t ldst;
};
hipError_t launch_quantize_fp8(const QuantFp8Args& a, hipStream_t stream);

// --------------------------------------------------------------- fp8_gemm.hip
struct GemmFp8Args {
  const uint8_t* a;  // [m, k]
  int64_t lda;
  const float* sa;  // [k / 128, m]
  int64_t ldsa;
  const uint8_t* b;  // [n, k]
  int64_t ldb;
  const float* sb;  // [n / 128, k / 128], or with b_rows [k / 128, n]
  int64_t ldsb;
  int b_rows;
  int64_t m, n, k;
  void* c;  // [m, n]
  int c_bf16;
  int64_t ldc;
  float* part;  // qgemm_fp8_partial_bytes() bytes
};
hipError_t launch_qgemm_fp8(const GemmFp8Args& a, hipStream_t stream);
int64_t qgemm_fp8_partial_bytes(int64_t m, int64_t n, int64_t k, bool c_bf16);

}  // namespace tp
