// C ABI of the rotated, quantized projection library (declared in
// include/tp.h). Every argument is validated here before any HIP call, so a
// refused call has enqueued no work (the TensorFold pull request #948 review
// asks for sizes and products to be checked before any device work; kvad-gpu
// internals, "Quantised weights on the GPU", refuses dimensions not divisible
// by 256 up front rather than failing halfway).
#include <hip/hip_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/tp.h"
#include "block_ops.hpp"
#include "kernels.hpp"

namespace {

thread_local char g_msg[512] = "";

tp_status fail(tp_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
tp_status fail(tp_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return st;
}

tp_status ok() {
  g_msg[0] = '\0';
  return TP_OK;
}

tp_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(TP_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }
bool add_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_add_overflow(a, b, out); }

// Byte extent [p, p + bytes) of a row-major matrix: (rows-1)*pitch + row_bytes.
struct Extent {
  uintptr_t lo = 0, hi = 0;
};

Extent extent_of(const void* p, int64_t rows, int64_t pitch_bytes, int64_t row_bytes) {
  Extent e;
  e.lo = (uintptr_t)p;
  e.hi = rows > 0 ? e.lo + (uintptr_t)((rows - 1) * pitch_bytes + row_bytes) : e.lo;
  return e;
}

bool overlaps(const Extent& a, const Extent& b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

int64_t dtype_size(tp_dtype d) { return d == TP_BF16 ? 2 : 4; }
bool dtype_ok(int d) { return d == TP_F32 || d == TP_BF16; }

// Validate one row-major operand: non-null (unless it is empty), ld >= row
// length, base and pitch aligned to `align` bytes, total extent representable.
// On success stores the extent (empty for an empty operand).
tp_status check_matrix(const char* name, const void* p, int64_t rows, int64_t cols_bytes, int64_t ld,
                       int64_t elem_bytes, Extent* ext, int64_t align = 16) {
  int64_t pitch;
  if (!mul_ok(ld, elem_bytes, &pitch)) return fail(TP_ERR_SIZE_OVERFLOW, "%s: ld * element size overflows", name);
  if (ld < 0 || pitch < cols_bytes)
    return fail(TP_ERR_BAD_LEADING_DIM, "%s: leading dimension %lld is smaller than the row (%lld bytes)", name,
                (long long)ld, (long long)cols_bytes);
  if (rows == 0 || cols_bytes == 0) {  // empty: nothing is read or written
    *ext = Extent{};
    return TP_OK;
  }
  if (!p) return fail(TP_ERR_NULL_POINTER, "%s is NULL", name);
  int64_t span;
  if (!mul_ok(rows - 1, pitch, &span) || !add_ok(span, cols_bytes, &span))
    return fail(TP_ERR_SIZE_OVERFLOW, "%s: byte extent overflows", name);
  if (((uintptr_t)p % (uintptr_t)align) != 0)
    return fail(TP_ERR_MISALIGNED, "%s: base pointer is not %lld-byte aligned", name, (long long)align);
  if (pitch % align != 0)
    return fail(TP_ERR_MISALIGNED, "%s: row pitch of %lld bytes is not a multiple of %lld", name, (long long)pitch,
                (long long)align);
  *ext = extent_of(p, rows, pitch, cols_bytes);
  return TP_OK;
}

tp_status check_vector(const char* name, const void* p, int64_t count, Extent* ext) {
  if (count == 0) {
    *ext = Extent{};
    return TP_OK;
  }
  if (!p) return fail(TP_ERR_NULL_POINTER, "%s is NULL", name);
  if (((uintptr_t)p & 3u) != 0) return fail(TP_ERR_MISALIGNED, "%s: not 4-byte aligned", name);
  int64_t bytes;
  if (!mul_ok(count, 4, &bytes)) return fail(TP_ERR_SIZE_OVERFLOW, "%s: size overflows", name);
  ext->lo = (uintptr_t)p;
  ext->hi = ext->lo + (uintptr_t)bytes;
  return TP_OK;
}

tp_status check_sizes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0) return fail(TP_ERR_BAD_SHAPE, "negative size (m=%lld, n=%lld)", (long long)m, (long long)n);
  if (k <= 0) return fail(TP_ERR_BAD_SHAPE, "k must be positive (k=%lld)", (long long)k);
  if (k % 256 != 0)
    return fail(TP_ERR_K_NOT_MULTIPLE_OF_256, "k=%lld is not a multiple of 256 (the rotation group)", (long long)k);
  if (m > INT_MAX || n > INT_MAX || k > INT_MAX)
    return fail(TP_ERR_BAD_SHAPE, "size above 2^31-1 (m=%lld, n=%lld, k=%lld)", (long long)m, (long long)n,
                (long long)k);
  return TP_OK;
}

#define TP_TRY(expr)                  \
  do {                                \
    tp_status _st = (expr);           \
    if (_st != TP_OK) return _st;     \
  } while (0)

int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// Workspace layout. Front part: W8/W4 with TP_A_ROTATE, bf16 A' [m, k];
// W8A8 (unless the caller takes the codes), int8 qa [m, k] then (256-byte
// aligned) fp32 sa [m]. Then, 256-byte aligned, the split-K partial sums of
// the small-M products (qgemm_partial_bytes; absent for larger M).
struct WsLayout {
  int64_t front = 0;     // bytes of the front part
  int64_t part_off = 0;  // offset of the partial sums
  int64_t total = 0;     // bytes needed
};

bool workspace_layout(tp_op op, int64_t m, int64_t n, int64_t k, int a_flags, bool own_codes, WsLayout* out) {
  int64_t mk;
  if (!mul_ok(m, k, &mk)) return false;
  int kind;
  WsLayout l;
  switch (op) {
    case TP_OP_QGEMM_W8:
    case TP_OP_QGEMM_W4:
      kind = op == TP_OP_QGEMM_W8 ? tp::GEMM_W8 : tp::GEMM_W4;
      if (a_flags == TP_A_ROTATE && !mul_ok(mk, 2, &l.front)) return false;
      break;
    case TP_OP_QGEMM_W8A8:
    case TP_OP_QGEMM_W4A8: {
      kind = op == TP_OP_QGEMM_W8A8 ? tp::GEMM_W8A8 : tp::GEMM_W4A8;
      if (!own_codes) {
        int64_t sa;
        if (!mul_ok(m, 4, &sa)) return false;
        if (mk > INT64_MAX - 512 - sa) return false;
        l.front = round_up(mk, 256) + sa;
      }
      break;
    }
    case TP_OP_QGEMM_W8A8_PREQUANTIZED:
      kind = tp::GEMM_W8A8;
      break;
    case TP_OP_QGEMM_W4A8_PREQUANTIZED:
      kind = tp::GEMM_W4A8;
      break;
    default:
      return false;
  }
  const int64_t part = tp::qgemm_partial_bytes(kind, m, n, k);
  if (part < 0 || l.front > INT64_MAX - 512 - part) return false;
  l.part_off = part > 0 ? round_up(l.front, 256) : l.front;
  l.total = l.part_off + part;
  *out = l;
  return true;
}

// Checks the caller's workspace against the layout; stores its extent.
tp_status check_workspace(const WsLayout& l, const void* ws, size_t ws_bytes, Extent* ew) {
  *ew = Extent{};
  if (l.total == 0) return TP_OK;
  if (!ws || (uint64_t)ws_bytes < (uint64_t)l.total)
    return fail(TP_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes given, %lld needed", ws_bytes,
                (long long)l.total);
  if (((uintptr_t)ws & 15u) != 0) return fail(TP_ERR_MISALIGNED, "workspace is not 16-byte aligned");
  ew->lo = (uintptr_t)ws;
  ew->hi = ew->lo + (uintptr_t)l.total;
  return TP_OK;
}

}  // namespace

extern "C" {

const char* tp_status_string(tp_status s) {
  switch (s) {
    case TP_OK: return "TP_OK";
    case TP_ERR_NULL_POINTER: return "TP_ERR_NULL_POINTER";
    case TP_ERR_BAD_SHAPE: return "TP_ERR_BAD_SHAPE";
    case TP_ERR_K_NOT_MULTIPLE_OF_256: return "TP_ERR_K_NOT_MULTIPLE_OF_256";
    case TP_ERR_BAD_LEADING_DIM: return "TP_ERR_BAD_LEADING_DIM";
    case TP_ERR_MISALIGNED: return "TP_ERR_MISALIGNED";
    case TP_ERR_UNSUPPORTED_DTYPE: return "TP_ERR_UNSUPPORTED_DTYPE";
    case TP_ERR_UNSUPPORTED_BITS: return "TP_ERR_UNSUPPORTED_BITS";
    case TP_ERR_SIZE_OVERFLOW: return "TP_ERR_SIZE_OVERFLOW";
    case TP_ERR_WORKSPACE_TOO_SMALL: return "TP_ERR_WORKSPACE_TOO_SMALL";
    case TP_ERR_BAD_ALIASING: return "TP_ERR_BAD_ALIASING";
    case TP_ERR_BAD_FLAGS: return "TP_ERR_BAD_FLAGS";
    case TP_ERR_HIP: return "TP_ERR_HIP";
    case TP_ERR_BAD_VALUE: return "TP_ERR_BAD_VALUE";
  }
  return "TP_ERR_UNKNOWN";
}

const char* tp_last_error_message(void) { return g_msg; }

int tp_abi_version(void) { return TP_ABI_VERSION; }

size_t tp_workspace_size(tp_op op, int64_t m, int64_t n, int64_t k, int a_flags) {
  if (m < 0 || n < 0 || k <= 0 || k % 256 != 0 || m > INT_MAX || n > INT_MAX || k > INT_MAX) return 0;
  WsLayout l;
  if (!workspace_layout(op, m, n, k, a_flags, false, &l)) return 0;
  return (size_t)l.total;
}

tp_status tp_rotate_quantize_weights(const void* w, tp_dtype w_dtype, int64_t n, int64_t k, int64_t ldw, int bits,
                                     void* q, int64_t ldq, float* scales, hipStream_t stream) {
  if (!dtype_ok(w_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "w_dtype %d is not TP_F32 or TP_BF16", (int)w_dtype);
  if (bits != 8 && bits != 4) return fail(TP_ERR_UNSUPPORTED_BITS, "bits=%d (expected 8 or 4)", bits);
  TP_TRY(check_sizes(0, n, k));
  Extent ew, eq, es;
  TP_TRY(check_matrix("w", w, n, k * dtype_size(w_dtype), ldw, dtype_size(w_dtype), &ew));
  TP_TRY(check_matrix("q", q, n, bits == 8 ? k : k / 2, ldq, 1, &eq));
  int64_t ns;
  if (!mul_ok(n, bits == 8 ? 1 : k / 256, &ns)) return fail(TP_ERR_SIZE_OVERFLOW, "scale count overflows");
  TP_TRY(check_vector("scales", scales, ns, &es));
  if (overlaps(ew, eq) || overlaps(ew, es) || overlaps(eq, es))
    return fail(TP_ERR_BAD_ALIASING, "w, q and scales must not overlap");
  if (n == 0) return ok();
  return hip_status(tp::launch_rotq_rows(w, w_dtype == TP_BF16, ldw, n, k, true, bits, q, ldq, scales, stream),
                    "rotate-quantize launch");
}

tp_status tp_hadamard_rotate_rows(const void* x, tp_dtype x_dtype, int64_t m, int64_t k, int64_t ldx, void* y,
                                  tp_dtype y_dtype, int64_t ldy, hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (!dtype_ok(y_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "y_dtype %d is not TP_F32 or TP_BF16", (int)y_dtype);
  TP_TRY(check_sizes(m, 0, k));
  Extent ex, ey;
  TP_TRY(check_matrix("x", x, m, k * dtype_size(x_dtype), ldx, dtype_size(x_dtype), &ex));
  TP_TRY(check_matrix("y", y, m, k * dtype_size(y_dtype), ldy, dtype_size(y_dtype), &ey));
  const bool in_place = (x == y && x_dtype == y_dtype && ldx == ldy);
  if (!in_place && overlaps(ex, ey))
    return fail(TP_ERR_BAD_ALIASING, "x and y overlap without being the same buffer, dtype and ld");
  if (m == 0) return ok();
  return hip_status(tp::launch_rotate_rows(x, x_dtype == TP_BF16, ldx, y, y_dtype == TP_BF16, ldy, m, k, stream),
                    "rotate launch");
}

tp_status tp_quantize_rows_int8(const void* x, tp_dtype x_dtype, int64_t m, int64_t k, int64_t ldx, int a_flags,
                                int8_t* qa, int64_t ldqa, float* sa, hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  TP_TRY(check_sizes(m, 0, k));
  Extent ex, eq, es;
  TP_TRY(check_matrix("x", x, m, k * dtype_size(x_dtype), ldx, dtype_size(x_dtype), &ex));
  TP_TRY(check_matrix("qa", qa, m, k, ldqa, 1, &eq));
  TP_TRY(check_vector("sa", sa, m, &es));
  if (overlaps(ex, eq) || overlaps(ex, es) || overlaps(eq, es))
    return fail(TP_ERR_BAD_ALIASING, "x, qa and sa must not overlap");
  if (m == 0) return ok();
  return hip_status(tp::launch_rotq_rows(x, x_dtype == TP_BF16, ldx, m, k, a_flags == TP_A_ROTATE, 8, qa, ldqa, sa,
                                         stream),
                    "activation quantize launch");
}

namespace {

tp_status check_codes(const char* name, const void* q, int bits, int64_t n, int64_t k, int64_t ldq, const char* sname,
                      const float* s, Extent* eq, Extent* es) {
  if (bits != 8 && bits != 4) return fail(TP_ERR_UNSUPPORTED_BITS, "%s: bits=%d is neither 8 nor 4", name, bits);
  TP_TRY(check_matrix(name, q, n, bits == 8 ? k : k / 2, ldq, 1, eq));
  int64_t ns;
  if (!mul_ok(n, bits == 8 ? 1 : k / 256, &ns)) return fail(TP_ERR_SIZE_OVERFLOW, "%s: scale count overflows", sname);
  return check_vector(sname, s, ns, es);
}

}  // namespace

size_t tp_lora_workspace_size(int64_t m, int64_t r) {
  if (m < 0 || r < 1 || r > 64 || m > INT_MAX) return 0;
  return (size_t)(m * 64 * 4);  // fp32 rows of 64 (zeros past r)
}

tp_status tp_lora_add(const void* x, tp_dtype x_dtype, int64_t ldx, const void* lora_a, const void* lora_b,
                      tp_dtype ab_dtype, int64_t lda, int64_t ldb, float alpha, int64_t m, int64_t n, int64_t k,
                      int64_t r, void* c, tp_dtype c_dtype, int64_t ldc, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (!dtype_ok(ab_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "ab_dtype %d is not TP_F32 or TP_BF16", (int)ab_dtype);
  if (!dtype_ok(c_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "c_dtype %d is not TP_F32 or TP_BF16", (int)c_dtype);
  TP_TRY(check_sizes(m, n, k));
  if (r < 1 || r > 64) return fail(TP_ERR_BAD_SHAPE, "rank r=%lld outside [1, 64]", (long long)r);
  const int64_t ex = dtype_size(x_dtype), eab = dtype_size(ab_dtype), ec_ = dtype_size(c_dtype);
  Extent e_x, e_a, e_b, e_c, e_w;
  TP_TRY(check_matrix("x", x, m, k * ex, ldx, ex, &e_x));
  TP_TRY(check_matrix("lora_a", lora_a, r, k * eab, lda, eab, &e_a));
  TP_TRY(check_matrix("lora_b", lora_b, n, r * eab, ldb, eab, &e_b));
  TP_TRY(check_matrix("c", c, m, n * ec_, ldc, ec_, &e_c, ec_));
  const int64_t need = m * 64 * 4;
  if (m > 0 && n > 0) {
    if (!workspace || (int64_t)workspace_bytes < need)
      return fail(TP_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %lld needed (tp_lora_workspace_size)",
                  workspace_bytes, (long long)need);
    if (((uintptr_t)workspace & 15u) != 0) return fail(TP_ERR_MISALIGNED, "workspace is not 16-byte aligned");
    e_w.lo = (uintptr_t)workspace;
    e_w.hi = e_w.lo + (uintptr_t)need;
  }
  const Extent* ins[] = {&e_x, &e_a, &e_b};
  for (const Extent* i : ins)
    if (overlaps(e_c, *i) || overlaps(e_w, *i)) return fail(TP_ERR_BAD_ALIASING, "c or the workspace overlaps an input");
  if (overlaps(e_c, e_w)) return fail(TP_ERR_BAD_ALIASING, "c and the workspace overlap");
  if (m == 0 || n == 0) return ok();
  return hip_status(tp::launch_lora_add(x, x_dtype == TP_BF16, ldx, lora_a, lora_b, ab_dtype == TP_BF16, lda, ldb,
                                        alpha, m, n, k, r, c, c_dtype == TP_BF16, ldc, (float*)workspace, stream),
                    "lora launch");
}

tp_status tp_lora_down(const void* x, tp_dtype x_dtype, int64_t ldx, const void* lora_a, tp_dtype a_dtype,
                       int64_t lda, int64_t m, int64_t k, int64_t r, float* t, size_t t_bytes, hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (!dtype_ok(a_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "a_dtype %d is not TP_F32 or TP_BF16", (int)a_dtype);
  TP_TRY(check_sizes(m, 0, k));
  if (r < 1 || r > 64) return fail(TP_ERR_BAD_SHAPE, "rank r=%lld outside [1, 64]", (long long)r);
  const int64_t ex = dtype_size(x_dtype), ea = dtype_size(a_dtype);
  Extent e_x, e_a, e_t;
  TP_TRY(check_matrix("x", x, m, k * ex, ldx, ex, &e_x));
  TP_TRY(check_matrix("lora_a", lora_a, r, k * ea, lda, ea, &e_a));
  if (m > 0 && (int64_t)t_bytes < m * 64 * 4)
    return fail(TP_ERR_WORKSPACE_TOO_SMALL, "t of %zu bytes, %lld needed (m rows of 64 floats)", t_bytes,
                (long long)(m * 64 * 4));
  TP_TRY(check_matrix("t", t, m, 64 * 4, 64, 4, &e_t));
  if (overlaps(e_t, e_x) || overlaps(e_t, e_a)) return fail(TP_ERR_BAD_ALIASING, "t overlaps an input");
  if (m == 0) return ok();
  return hip_status(tp::launch_lora_down(x, x_dtype == TP_BF16, ldx, lora_a, a_dtype == TP_BF16, lda, m, k, r, t,
                                         stream),
                    "lora down launch");
}

tp_status tp_dequantize_unrotate(const void* q, int bits, int64_t ldq_bytes, const float* scales, int64_t n,
                                 int64_t k, void* w, tp_dtype w_dtype, int64_t ldw, hipStream_t stream) {
  if (!dtype_ok(w_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "w_dtype %d is not TP_F32 or TP_BF16", (int)w_dtype);
  TP_TRY(check_sizes(0, n, k));
  Extent eq, es, ew;
  TP_TRY(check_codes("q", q, bits, n, k, ldq_bytes, "scales", scales, &eq, &es));
  TP_TRY(check_matrix("w", w, n, k * dtype_size(w_dtype), ldw, dtype_size(w_dtype), &ew));
  if (overlaps(ew, eq) || overlaps(ew, es)) return fail(TP_ERR_BAD_ALIASING, "w must not overlap q or scales");
  if (n == 0) return ok();
  return hip_status(tp::launch_dequant_unrotate(q, bits, ldq_bytes, scales, n, k, w, w_dtype == TP_BF16, ldw, stream),
                    "dequantize launch");
}

tp_status tp_requantize_weights(const void* q_in, int bits_in, int64_t ldq_in, const float* s_in, int64_t n,
                                int64_t k, int bits_out, void* q_out, int64_t ldq_out, float* s_out,
                                hipStream_t stream) {
  TP_TRY(check_sizes(0, n, k));
  Extent eqi, esi, eqo, eso;
  TP_TRY(check_codes("q_in", q_in, bits_in, n, k, ldq_in, "s_in", s_in, &eqi, &esi));
  TP_TRY(check_codes("q_out", q_out, bits_out, n, k, ldq_out, "s_out", s_out, &eqo, &eso));
  if (overlaps(eqo, eqi) || overlaps(eqo, esi) || overlaps(eso, eqi) || overlaps(eso, esi) || overlaps(eqo, eso))
    return fail(TP_ERR_BAD_ALIASING, "q_out and s_out must not overlap the inputs or each other");
  if (n == 0) return ok();
  return hip_status(tp::launch_requantize(q_in, bits_in, ldq_in, s_in, n, k, bits_out, q_out, ldq_out, s_out, stream),
                    "requantize launch");
}

tp_status tp_swiglu_rotate(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, tp_dtype in_dtype,
                           int64_t m, int64_t k, int out_kind, void* y, int64_t ldy, float* scales,
                           hipStream_t stream) {
  if (!dtype_ok(in_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "in_dtype %d is not TP_F32 or TP_BF16", (int)in_dtype);
  if (out_kind != TP_FFN_OUT_I8 && out_kind != TP_FFN_OUT_BF16) return fail(TP_ERR_BAD_FLAGS, "out_kind=%d", out_kind);
  TP_TRY(check_sizes(m, 0, k));
  const bool i8 = out_kind == TP_FFN_OUT_I8;
  const int64_t es = dtype_size(in_dtype), ys = i8 ? 1 : 2;
  Extent eg, eu, ey, esc;
  TP_TRY(check_matrix("gate", gate, m, k * es, ld_gate, es, &eg));
  TP_TRY(check_matrix("up", up, m, k * es, ld_up, es, &eu));
  TP_TRY(check_matrix("y", y, m, k * ys, ldy, ys, &ey));
  if (i8) {
    TP_TRY(check_vector("scales", scales, m, &esc));
    if (overlaps(esc, eg) || overlaps(esc, eu) || overlaps(esc, ey))
      return fail(TP_ERR_BAD_ALIASING, "scales must not overlap gate, up or y");
  }
  if (overlaps(ey, eg) || overlaps(ey, eu)) return fail(TP_ERR_BAD_ALIASING, "y must not overlap gate or up");
  if (m == 0) return ok();
  return hip_status(tp::launch_swiglu_rotate(gate, ld_gate, up, ld_up, in_dtype == TP_BF16, m, k, i8, y, ldy,
                                             i8 ? scales : nullptr, stream),
                    "swiglu rotate launch");
}

namespace {

// Shared by the two weight-only products.
tp_status weight_only(int kind, const void* a, tp_dtype a_dtype, int64_t lda, int a_flags, const void* q,
                      int64_t ldq, const float* w_scales, int64_t m, int64_t n, int64_t k, void* c, tp_dtype c_dtype,
                      int64_t ldc, void* ws, size_t ws_bytes, hipStream_t stream) {
  const tp_op op = kind == tp::GEMM_W8 ? TP_OP_QGEMM_W8 : TP_OP_QGEMM_W4;
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  if (!dtype_ok(a_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "a_dtype %d is not TP_F32 or TP_BF16", (int)a_dtype);
  if (a_flags == TP_A_PREROTATED && a_dtype != TP_BF16)
    return fail(TP_ERR_UNSUPPORTED_DTYPE, "a pre-rotated operand must be TP_BF16");
  if (!dtype_ok(c_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "c_dtype %d is not TP_F32 or TP_BF16", (int)c_dtype);
  TP_TRY(check_sizes(m, n, k));
  Extent ea, eq, es, ec, ew;
  TP_TRY(check_matrix("a", a, m, k * dtype_size(a_dtype), lda, dtype_size(a_dtype), &ea));
  TP_TRY(check_matrix("q", q, n, kind == tp::GEMM_W8 ? k : k / 2, ldq, 1, &eq));
  int64_t ns;
  if (!mul_ok(n, kind == tp::GEMM_W8 ? 1 : k / 256, &ns)) return fail(TP_ERR_SIZE_OVERFLOW, "scale count overflows");
  TP_TRY(check_vector("w_scales", w_scales, ns, &es));
  TP_TRY(check_matrix("c", c, m, n * dtype_size(c_dtype), ldc, dtype_size(c_dtype), &ec, dtype_size(c_dtype)));
  WsLayout wl;
  if (!workspace_layout(op, m, n, k, a_flags, false, &wl)) return fail(TP_ERR_SIZE_OVERFLOW, "workspace size overflows");
  TP_TRY(check_workspace(wl, ws, ws_bytes, &ew));
  if (overlaps(ec, ea) || overlaps(ec, eq) || overlaps(ec, es) || overlaps(ec, ew) || overlaps(ew, ea) ||
      overlaps(ew, eq) || overlaps(ew, es))
    return fail(TP_ERR_BAD_ALIASING, "c and the workspace must not overlap any other operand");
  if (m == 0 || n == 0) return ok();

  const void* a_rot = a;
  int64_t lda_rot = lda;
  if (a_flags == TP_A_ROTATE) {
    TP_TRY(hip_status(tp::launch_rotate_rows(a, a_dtype == TP_BF16, lda, ws, true, k, m, k, stream), "rotate launch"));
    a_rot = ws;
    lda_rot = k;
  }
  tp::GemmArgs g{};
  g.kind = kind;
  g.a = a_rot;
  g.lda = lda_rot;
  g.b = q;
  g.ldb = ldq;
  g.w_scales = w_scales;
  g.a_scales = nullptr;
  g.m = m;
  g.n = n;
  g.k = k;
  g.c = c;
  g.c_bf16 = c_dtype == TP_BF16;
  g.ldc = ldc;
  g.acc_out = nullptr;
  g.ld_acc = 0;
  g.part = wl.total > wl.part_off ? (uint8_t*)ws + wl.part_off : nullptr;
  return hip_status(tp::launch_qgemm(g, stream), "product launch");
}

}  // namespace

tp_status tp_qgemm_w8(const void* a, tp_dtype a_dtype, int64_t lda, int a_flags, const int8_t* q, int64_t ldq,
                      const float* w_scales, int64_t m, int64_t n, int64_t k, void* c, tp_dtype c_dtype, int64_t ldc,
                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return weight_only(tp::GEMM_W8, a, a_dtype, lda, a_flags, q, ldq, w_scales, m, n, k, c, c_dtype, ldc, workspace,
                     workspace_bytes, stream);
}

tp_status tp_qgemm_w4(const void* a, tp_dtype a_dtype, int64_t lda, int a_flags, const uint8_t* q, int64_t ldq,
                      const float* w_scales, int64_t m, int64_t n, int64_t k, void* c, tp_dtype c_dtype, int64_t ldc,
                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return weight_only(tp::GEMM_W4, a, a_dtype, lda, a_flags, q, ldq, w_scales, m, n, k, c, c_dtype, ldc, workspace,
                     workspace_bytes, stream);
}

namespace {

// The int8 x int8 (W8A8) and int8 x int4 (W4A8) products on activations the
// library quantizes first. acc_out is W8A8 only.
tp_status act8_product(int kind, const void* a, tp_dtype a_dtype, int64_t lda, int a_flags, const void* q,
                       int64_t ldq, const float* w_scales, int64_t m, int64_t n, int64_t k, void* c,
                       tp_dtype c_dtype, int64_t ldc, int8_t* qa_out, float* sa_out, int32_t* acc_out,
                       int64_t ld_acc, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool w4 = kind == tp::GEMM_W4A8;
  const tp_op op = w4 ? TP_OP_QGEMM_W4A8 : TP_OP_QGEMM_W8A8;
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  if (!dtype_ok(a_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "a_dtype %d is not TP_F32 or TP_BF16", (int)a_dtype);
  if (!dtype_ok(c_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "c_dtype %d is not TP_F32 or TP_BF16", (int)c_dtype);
  TP_TRY(check_sizes(m, n, k));
  if (!w4 && k > INT32_MAX / (127 * 127))
    return fail(TP_ERR_BAD_SHAPE, "k=%lld: the int32 accumulator could overflow (k <= %d)", (long long)k,
                INT32_MAX / (127 * 127));
  Extent ea, eq, es, ec, eqa, esa, eacc, ew;
  TP_TRY(check_matrix("a", a, m, k * dtype_size(a_dtype), lda, dtype_size(a_dtype), &ea));
  TP_TRY(check_matrix("q", q, n, w4 ? k / 2 : k, ldq, 1, &eq));
  int64_t ns;
  if (!mul_ok(n, w4 ? k / 256 : 1, &ns)) return fail(TP_ERR_SIZE_OVERFLOW, "scale count overflows");
  TP_TRY(check_vector("w_scales", w_scales, ns, &es));
  TP_TRY(check_matrix("c", c, m, n * dtype_size(c_dtype), ldc, dtype_size(c_dtype), &ec, dtype_size(c_dtype)));
  const bool own_codes = qa_out && sa_out;
  if (qa_out) TP_TRY(check_matrix("qa_out", qa_out, m, k, k, 1, &eqa));
  if (sa_out) TP_TRY(check_vector("sa_out", sa_out, m, &esa));
  if (acc_out) TP_TRY(check_matrix("acc_out", acc_out, m, n * 4, ld_acc, 4, &eacc, 4));
  WsLayout wl;
  if (!workspace_layout(op, m, n, k, a_flags, own_codes, &wl))
    return fail(TP_ERR_SIZE_OVERFLOW, "workspace size overflows");
  TP_TRY(check_workspace(wl, workspace, workspace_bytes, &ew));
  const Extent* outs[] = {&ec, &eqa, &esa, &eacc, &ew};
  const Extent* ins[] = {&ea, &eq, &es};
  for (const Extent* o : outs) {
    for (const Extent* i : ins)
      if (overlaps(*o, *i)) return fail(TP_ERR_BAD_ALIASING, "an output or the workspace overlaps an input");
    for (const Extent* o2 : outs)
      if (o2 != o && overlaps(*o, *o2)) return fail(TP_ERR_BAD_ALIASING, "two outputs overlap");
  }
  if (m == 0 || n == 0) return ok();

  int8_t* qa = qa_out ? qa_out : (int8_t*)workspace;
  float* sa = sa_out ? sa_out : (float*)((uint8_t*)workspace + round_up(m * k, 256));
  TP_TRY(hip_status(tp::launch_rotq_rows(a, a_dtype == TP_BF16, lda, m, k, a_flags == TP_A_ROTATE, 8, qa, k, sa,
                                         stream),
                    "activation quantize launch"));
  tp::GemmArgs g{};
  g.kind = kind;
  g.a = qa;
  g.lda = k;
  g.b = q;
  g.ldb = ldq;
  g.w_scales = w_scales;
  g.a_scales = sa;
  g.m = m;
  g.n = n;
  g.k = k;
  g.c = c;
  g.c_bf16 = c_dtype == TP_BF16;
  g.ldc = ldc;
  g.acc_out = acc_out;
  g.ld_acc = ld_acc;
  g.part = wl.total > wl.part_off ? (uint8_t*)workspace + wl.part_off : nullptr;
  return hip_status(tp::launch_qgemm(g, stream), "product launch");
}

// The side path of tp_qgemm_w8a8_prequantized_lora: T fp32 [m, 64] (rows of
// 64 floats, zeros past r) and lora_b bf16 [n, r]; fp32 C only.
struct LoraIn {
  const float* t;
  const void* b;
  int64_t ldb;
  int64_t r;
  float alpha;
};

tp_status prequantized_product(int kind, const int8_t* qa, int64_t ldqa, const float* sa, const void* q, int64_t ldq,
                               const float* w_scales, int64_t m, int64_t n, int64_t k, void* c, tp_dtype c_dtype,
                               int64_t ldc, int32_t* acc_out, int64_t ld_acc, void* workspace,
                               size_t workspace_bytes, hipStream_t stream, const LoraIn* lora = nullptr,
                               bool noalloc = false) {
  const bool w4 = kind == tp::GEMM_W4A8;
  const tp_op op = w4 ? TP_OP_QGEMM_W4A8_PREQUANTIZED : TP_OP_QGEMM_W8A8_PREQUANTIZED;
  if (!dtype_ok(c_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "c_dtype %d is not TP_F32 or TP_BF16", (int)c_dtype);
  TP_TRY(check_sizes(m, n, k));
  if (!w4 && k > INT32_MAX / (127 * 127))
    return fail(TP_ERR_BAD_SHAPE, "k=%lld: the int32 accumulator could overflow (k <= %d)", (long long)k,
                INT32_MAX / (127 * 127));
  Extent eqa, esa, eq, es, ec, eacc;
  TP_TRY(check_matrix("qa", qa, m, k, ldqa, 1, &eqa));
  TP_TRY(check_vector("sa", sa, m, &esa));
  TP_TRY(check_matrix("q", q, n, w4 ? k / 2 : k, ldq, 1, &eq));
  int64_t ns;
  if (!mul_ok(n, w4 ? k / 256 : 1, &ns)) return fail(TP_ERR_SIZE_OVERFLOW, "scale count overflows");
  TP_TRY(check_vector("w_scales", w_scales, ns, &es));
  TP_TRY(check_matrix("c", c, m, n * dtype_size(c_dtype), ldc, dtype_size(c_dtype), &ec, dtype_size(c_dtype)));
  if (acc_out) TP_TRY(check_matrix("acc_out", acc_out, m, n * 4, ld_acc, 4, &eacc, 4));
  Extent et, eb;
  if (lora) {
    if (c_dtype != TP_F32) return fail(TP_ERR_UNSUPPORTED_DTYPE, "the side path adds into fp32 C only");
    if (lora->r < 1 || lora->r > 64) return fail(TP_ERR_BAD_SHAPE, "rank r=%lld outside [1, 64]", (long long)lora->r);
    TP_TRY(check_matrix("t", lora->t, m, 64 * 4, 64, 4, &et));
    TP_TRY(check_matrix("lora_b", lora->b, n, lora->r * 2, lora->ldb, 2, &eb));
  }
  WsLayout wl;
  Extent ew;
  if (!workspace_layout(op, m, n, k, TP_A_PREROTATED, true, &wl))
    return fail(TP_ERR_SIZE_OVERFLOW, "workspace size overflows");
  if (noalloc) {
    // the library's own scratch array instead of a workspace (no overlap with
    // any caller buffer possible)
    if (wl.total > tp::NOALLOC_SCRATCH_BYTES)
      return fail(TP_ERR_WORKSPACE_TOO_SMALL,
                  "this shape needs %lld bytes of split-K partial sums; the no-allocation entry point holds %lld "
                  "(use tp_qgemm_w8a8_prequantized with a workspace)",
                  (long long)wl.total, (long long)tp::NOALLOC_SCRATCH_BYTES);
  } else {
    TP_TRY(check_workspace(wl, workspace, workspace_bytes, &ew));
  }
  const Extent* ins[] = {&eqa, &esa, &eq, &es, &et, &eb};
  for (const Extent* i : ins)
    if (overlaps(ec, *i) || overlaps(eacc, *i) || overlaps(ew, *i))
      return fail(TP_ERR_BAD_ALIASING, "an output or the workspace overlaps an input");
  if (overlaps(ec, eacc) || overlaps(ec, ew) || overlaps(eacc, ew))
    return fail(TP_ERR_BAD_ALIASING, "c, acc_out and the workspace must not overlap");
  if (m == 0 || n == 0) return ok();
  tp::GemmArgs g{};
  g.kind = kind;
  g.a = qa;
  g.lda = ldqa;
  g.b = q;
  g.ldb = ldq;
  g.w_scales = w_scales;
  g.a_scales = sa;
  g.m = m;
  g.n = n;
  g.k = k;
  g.c = c;
  g.c_bf16 = c_dtype == TP_BF16;
  g.ldc = ldc;
  g.acc_out = acc_out;
  g.ld_acc = ld_acc;
  g.part = wl.total > 0 ? workspace : nullptr;
  if (noalloc && wl.total > 0) TP_TRY(hip_status(tp::noalloc_scratch(&g.part), "scratch address"));
  if (lora) {
    g.lora.t = lora->t;
    g.lora.b = (const uint16_t*)lora->b;
    g.lora.ldb = lora->ldb;
    g.lora.r = (int)lora->r;
    g.lora.alpha = lora->alpha;
  }
  return hip_status(tp::launch_qgemm(g, stream), "product launch");
}

}  // namespace

tp_status tp_qgemm_w8a8(const void* a, tp_dtype a_dtype, int64_t lda, int a_flags, const int8_t* q, int64_t ldq,
                        const float* w_scales, int64_t m, int64_t n, int64_t k, void* c, tp_dtype c_dtype,
                        int64_t ldc, int8_t* qa_out, float* sa_out, int32_t* acc_out, int64_t ld_acc,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return act8_product(tp::GEMM_W8A8, a, a_dtype, lda, a_flags, q, ldq, w_scales, m, n, k, c, c_dtype, ldc, qa_out,
                      sa_out, acc_out, ld_acc, workspace, workspace_bytes, stream);
}

tp_status tp_qgemm_w8a8_prequantized(const int8_t* qa, int64_t ldqa, const float* sa, const int8_t* q, int64_t ldq,
                                     const float* w_scales, int64_t m, int64_t n, int64_t k, void* c,
                                     tp_dtype c_dtype, int64_t ldc, int32_t* acc_out, int64_t ld_acc,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return prequantized_product(tp::GEMM_W8A8, qa, ldqa, sa, q, ldq, w_scales, m, n, k, c, c_dtype, ldc, acc_out,
                              ld_acc, workspace, workspace_bytes, stream);
}

tp_status tp_qgemm_w8a8_prequantized_noalloc(const int8_t* qa, int64_t ldqa, const float* sa, const int8_t* q,
                                             int64_t ldq, const float* w_scales, int64_t m, int64_t n, int64_t k,
                                             void* c, tp_dtype c_dtype, int64_t ldc, int32_t* acc_out,
                                             int64_t ld_acc, hipStream_t stream) {
  return prequantized_product(tp::GEMM_W8A8, qa, ldqa, sa, q, ldq, w_scales, m, n, k, c, c_dtype, ldc, acc_out,
                              ld_acc, nullptr, 0, stream, nullptr, true);
}

tp_status tp_qgemm_w8a8_prequantized_lora(const int8_t* qa, int64_t ldqa, const float* sa, const int8_t* q,
                                          int64_t ldq, const float* w_scales, int64_t m, int64_t n, int64_t k,
                                          float* c, int64_t ldc, const float* t, const void* lora_b, int64_t ldb,
                                          int64_t r, float alpha, void* workspace, size_t workspace_bytes,
                                          hipStream_t stream) {
  const LoraIn lora{t, lora_b, ldb, r, alpha};
  return prequantized_product(tp::GEMM_W8A8, qa, ldqa, sa, q, ldq, w_scales, m, n, k, c, TP_F32, ldc, nullptr, 0,
                              workspace, workspace_bytes, stream, &lora);
}

tp_status tp_qgemm_w4a8(const void* a, tp_dtype a_dtype, int64_t lda, int a_flags, const uint8_t* q4,
                        int64_t ldq_bytes, const float* w_scales, int64_t m, int64_t n, int64_t k, void* c,
                        tp_dtype c_dtype, int64_t ldc, int8_t* qa_out, float* sa_out, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  return act8_product(tp::GEMM_W4A8, a, a_dtype, lda, a_flags, q4, ldq_bytes, w_scales, m, n, k, c, c_dtype, ldc,
                      qa_out, sa_out, nullptr, 0, workspace, workspace_bytes, stream);
}

tp_status tp_qgemm_w4a8_prequantized(const int8_t* qa, int64_t ldqa, const float* sa, const uint8_t* q4,
                                     int64_t ldq_bytes, const float* w_scales, int64_t m, int64_t n, int64_t k,
                                     void* c, tp_dtype c_dtype, int64_t ldc, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  return prequantized_product(tp::GEMM_W4A8, qa, ldqa, sa, q4, ldq_bytes, w_scales, m, n, k, c, c_dtype, ldc,
                              nullptr, 0, workspace, workspace_bytes, stream);
}

// ------------------------------------------------ norm around the projections

namespace {

// (below 1e-30 the factor of a row of zeros and its cube leave fp32: zeros would
// come out as NaN)
tp_status check_eps(double eps) {
  if (!(eps >= 1e-30) || !(eps <= 1e30)) return fail(TP_ERR_BAD_VALUE, "eps=%g is not within 1e-30 .. 1e30", eps);
  return TP_OK;
}

// A weight vector: optional, contiguous, 16-byte aligned.
tp_status check_weight(const char* name, const void* p, tp_dtype dtype, int64_t count, Extent* ext) {
  *ext = Extent{};
  if (!p) return TP_OK;
  if (!dtype_ok(dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "%s: dtype %d is not TP_F32 or TP_BF16", name, (int)dtype);
  return check_matrix(name, p, 1, count * dtype_size(dtype), count, dtype_size(dtype), ext);
}

tp_status check_norm_k(int64_t k) {
  if (k / 256 > tp::NORM_MAX_GROUPS)
    return fail(TP_ERR_BAD_SHAPE, "k=%lld: rows of at most %d columns", (long long)k, tp::NORM_MAX_GROUPS * 256);
  return TP_OK;
}

// Whether out may be the very buffer of in.
bool same_buffer(const void* out, tp_dtype od, int64_t ldo, const void* in, tp_dtype id, int64_t ldi) {
  return out == in && od == id && ldo == ldi;
}

// The caller's scratch memory, where `need` bytes of it are used.
tp_status check_scratch(const char* query, const void* ws, size_t ws_bytes, int64_t need, Extent* ew) {
  *ew = Extent{};
  if (need == 0) return TP_OK;
  if (!ws || (uint64_t)ws_bytes < (uint64_t)need)
    return fail(TP_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %lld needed (%s)", ws_bytes, (long long)need, query);
  if (((uintptr_t)ws & 15u) != 0) return fail(TP_ERR_MISALIGNED, "workspace is not 16-byte aligned");
  ew->lo = (uintptr_t)ws;
  ew->hi = ew->lo + (uintptr_t)need;
  return TP_OK;
}

}  // namespace

tp_status tp_rmsnorm_rotate(const void* x, tp_dtype x_dtype, int64_t ldx, const void* residual, int64_t ldr,
                            void* sum_out, int64_t ldsum, tp_dtype s_dtype, const void* gamma, tp_dtype g_dtype,
                            double eps, int a_flags, int64_t m, int64_t k, int out_kind, void* y, int64_t ldy,
                            float* scales, hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (out_kind != TP_NORM_OUT_I8 && out_kind != TP_NORM_OUT_BF16) return fail(TP_ERR_BAD_FLAGS, "out_kind=%d", out_kind);
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  TP_TRY(check_sizes(m, 0, k));
  TP_TRY(check_norm_k(k));
  TP_TRY(check_eps(eps));
  const bool i8 = out_kind == TP_NORM_OUT_I8;
  const int64_t xs = dtype_size(x_dtype);
  Extent ex, er{}, esum{}, eg, ey, esc{};
  TP_TRY(check_matrix("x", x, m, k * xs, ldx, xs, &ex));
  if (residual || sum_out) {
    if (!dtype_ok(s_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "s_dtype %d is not TP_F32 or TP_BF16", (int)s_dtype);
    const int64_t ss = dtype_size(s_dtype);
    if (!residual || !sum_out)
      return fail(TP_ERR_NULL_POINTER, "residual and sum_out are given together or not at all");
    TP_TRY(check_matrix("residual", residual, m, k * ss, ldr, ss, &er));
    TP_TRY(check_matrix("sum_out", sum_out, m, k * ss, ldsum, ss, &esum));
  }
  TP_TRY(check_weight("gamma", gamma, g_dtype, k, &eg));
  TP_TRY(check_matrix("y", y, m, k * (i8 ? 1 : 2), ldy, i8 ? 1 : 2, &ey));
  if (i8) TP_TRY(check_vector("scales", scales, m, &esc));
  const Extent* outs[] = {&ey, &esc};
  for (const Extent* o : outs)
    if (overlaps(*o, ex) || overlaps(*o, er) || overlaps(*o, esum) || overlaps(*o, eg))
      return fail(TP_ERR_BAD_ALIASING, "y and scales must not overlap x, residual, sum_out or gamma");
  if (overlaps(ey, esc)) return fail(TP_ERR_BAD_ALIASING, "y and scales overlap");
  if (overlaps(esum, eg)) return fail(TP_ERR_BAD_ALIASING, "sum_out overlaps gamma");
  if (overlaps(esum, er) && !same_buffer(sum_out, s_dtype, ldsum, residual, s_dtype, ldr))
    return fail(TP_ERR_BAD_ALIASING, "sum_out overlaps residual without being the same buffer");
  if (overlaps(esum, ex) && !same_buffer(sum_out, s_dtype, ldsum, x, x_dtype, ldx))
    return fail(TP_ERR_BAD_ALIASING, "sum_out overlaps x without being the same buffer");
  if (m == 0) return ok();
  tp::NormArgs a{};
  a.x = x;
  a.x_bf16 = x_dtype == TP_BF16;
  a.ldx = ldx;
  a.res = residual;
  a.ldr = ldr;
  a.sum = sum_out;
  a.ldsum = ldsum;
  a.s_bf16 = residual && s_dtype == TP_BF16;
  a.gamma = {gamma, gamma && g_dtype == TP_BF16};
  a.eps = eps;
  a.rotate = a_flags == TP_A_ROTATE;
  a.m = m;
  a.groups = (int)(k / 256);
  a.out_i8 = i8;
  a.y = y;
  a.ldy = ldy;
  a.scales = i8 ? scales : nullptr;
  return hip_status(tp::launch_norm_rotate(a, stream), "norm launch");
}

size_t tp_rmsnorm_backward_workspace_size(int64_t m, int64_t k) {
  if (m <= 0 || k <= 0 || k % 256 != 0 || m > INT_MAX || k / 256 > tp::NORM_MAX_GROUPS) return 0;
  return (size_t)(tp::norm_bwd_partial_rows(m, (int)(k / 256)) * k * 4);
}

tp_status tp_rmsnorm_rotate_backward(const void* dy, tp_dtype dy_dtype, int64_t lddy, int a_flags, const void* t,
                                     tp_dtype t_dtype, int64_t ldt, const void* gamma, tp_dtype g_dtype, double eps,
                                     const void* dsum, int64_t ldds, int64_t m, int64_t k, void* dx,
                                     tp_dtype dx_dtype, int64_t lddx, float* dgamma, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dy_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "dy_dtype %d is not TP_F32 or TP_BF16", (int)dy_dtype);
  if (!dtype_ok(t_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "t_dtype %d is not TP_F32 or TP_BF16", (int)t_dtype);
  if (!dtype_ok(dx_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "dx_dtype %d is not TP_F32 or TP_BF16", (int)dx_dtype);
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  TP_TRY(check_sizes(m, 0, k));
  TP_TRY(check_norm_k(k));
  TP_TRY(check_eps(eps));
  const int64_t gs = dtype_size(dy_dtype), ts = dtype_size(t_dtype), xs = dtype_size(dx_dtype);
  Extent edy, et, eg, eds{}, edx, edg{}, ew;
  TP_TRY(check_matrix("dy", dy, m, k * gs, lddy, gs, &edy));
  TP_TRY(check_matrix("t", t, m, k * ts, ldt, ts, &et));
  TP_TRY(check_weight("gamma", gamma, g_dtype, k, &eg));
  if (dsum) TP_TRY(check_matrix("dsum", dsum, m, k * xs, ldds, xs, &eds));
  TP_TRY(check_matrix("dx", dx, m, k * xs, lddx, xs, &edx));
  if (dgamma) TP_TRY(check_vector("dgamma", dgamma, k, &edg));
  TP_TRY(check_scratch("tp_rmsnorm_backward_workspace_size", workspace, workspace_bytes,
                       dgamma ? (int64_t)tp_rmsnorm_backward_workspace_size(m, k) : 0, &ew));
  const Extent* ins[] = {&edy, &et, &eg, &eds};
  for (const Extent* i : ins)
    if (overlaps(edg, *i) || overlaps(ew, *i))
      return fail(TP_ERR_BAD_ALIASING, "dgamma or the workspace overlaps an input");
  if (overlaps(edx, edg) || overlaps(edx, ew) || overlaps(edg, ew))
    return fail(TP_ERR_BAD_ALIASING, "dx, dgamma and the workspace must not overlap");
  if (overlaps(edx, et) || overlaps(edx, eg)) return fail(TP_ERR_BAD_ALIASING, "dx overlaps t or gamma");
  if (overlaps(edx, eds) && !same_buffer(dx, dx_dtype, lddx, dsum, dx_dtype, ldds))
    return fail(TP_ERR_BAD_ALIASING, "dx overlaps dsum without being the same buffer");
  if (overlaps(edx, edy) && !same_buffer(dx, dx_dtype, lddx, dy, dy_dtype, lddy))
    return fail(TP_ERR_BAD_ALIASING, "dx overlaps dy without being the same buffer");
  if (m == 0 && !dgamma) return ok();
  tp::NormBwdArgs a{};
  a.dy = dy;
  a.dy_bf16 = dy_dtype == TP_BF16;
  a.lddy = lddy;
  a.rotate = a_flags == TP_A_ROTATE;
  a.t = t;
  a.t_bf16 = t_dtype == TP_BF16;
  a.ldt = ldt;
  a.gamma = {gamma, gamma && g_dtype == TP_BF16};
  a.eps = eps;
  a.dsum = dsum;
  a.ldds = ldds;
  a.m = m;
  a.groups = (int)(k / 256);
  a.dx = dx;
  a.dx_bf16 = dx_dtype == TP_BF16;
  a.lddx = lddx;
  a.dgamma = dgamma;
  a.part = (float*)workspace;
  return hip_status(tp::launch_norm_bwd(a, stream), "norm backward launch");
}

// ------------------------------------------- side path on 8-bit activations

namespace {

// Rows and columns: a launch counts its threads in 32 bits, and the most threads
// an element (32 for a row's planes and for 64 ranks of a column of A) stay below.
constexpr int64_t SIDE_MAX = (int64_t)1 << 26;

tp_status check_rank(int64_t r) {
  if (r < 1 || r > 64) return fail(TP_ERR_BAD_SHAPE, "rank r=%lld outside [1, 64]", (long long)r);
  return TP_OK;
}

}  // namespace

size_t tp_lora_down_prequantized_workspace_size(int64_t m, int64_t k, int64_t r) {
  if (m < 0 || m >= SIDE_MAX || k <= 0 || k % 256 != 0 || k > INT_MAX || r < 1 || r > 64) return 0;
  return (size_t)(tp::side_down_workspace_floats(m, k, r) * 4);
}

tp_status tp_lora_down_prequantized(const int8_t* qa, int64_t ldqa, const float* sa, const void* lora_a,
                                    tp_dtype a_dtype, int64_t lda, int64_t m, int64_t k, int64_t r, float* t,
                                    size_t t_bytes, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(a_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "a_dtype %d is not TP_F32 or TP_BF16", (int)a_dtype);
  TP_TRY(check_sizes(m, 0, k));
  TP_TRY(check_rank(r));
  if (m >= SIDE_MAX) return fail(TP_ERR_BAD_SHAPE, "m=%lld: below 2^26", (long long)m);
  const int64_t as = dtype_size(a_dtype);
  Extent eq, es, ea, et, ew;
  TP_TRY(check_matrix("qa", qa, m, k, ldqa, 1, &eq));
  TP_TRY(check_vector("sa", sa, m, &es));
  TP_TRY(check_matrix("lora_a", lora_a, r, k * as, lda, as, &ea));
  if (m > 0 && (uint64_t)t_bytes < (uint64_t)(m * 64 * 4))
    return fail(TP_ERR_WORKSPACE_TOO_SMALL, "t of %zu bytes, %lld needed (m rows of 64 floats)", t_bytes,
                (long long)(m * 64 * 4));
  TP_TRY(check_matrix("t", t, m, 64 * 4, 64, 4, &et));
  TP_TRY(check_scratch("tp_lora_down_prequantized_workspace_size", workspace, workspace_bytes,
                       (int64_t)tp_lora_down_prequantized_workspace_size(m, k, r), &ew));
  const Extent* ins[] = {&eq, &es, &ea};
  for (const Extent* i : ins)
    if (overlaps(et, *i) || overlaps(ew, *i)) return fail(TP_ERR_BAD_ALIASING, "t or the workspace overlaps an input");
  if (overlaps(et, ew)) return fail(TP_ERR_BAD_ALIASING, "t and the workspace overlap");
  if (m == 0) return ok();
  tp::SideDownArgs a{};
  a.qa = qa;
  a.ldqa = ldqa;
  a.sa = sa;
  a.a = lora_a;
  a.a_bf16 = a_dtype == TP_BF16;
  a.lda = lda;
  a.m = m;
  a.k = k;
  a.r = (int)r;
  a.t = t;
  a.ws = (float*)workspace;
  return hip_status(tp::launch_side_down(a, stream), "side path launch");
}

size_t tp_lora_grad_workspace_size(int64_t m, int64_t n, int64_t k, int64_t r) {
  if (m < 0 || n < 0 || m >= SIDE_MAX || n >= SIDE_MAX || k <= 0 || k % 256 != 0 || k >= SIDE_MAX || r < 1 || r > 64)
    return 0;
  return (size_t)(tp::side_grad_workspace_floats(m, n, k, r) * 4);
}

tp_status tp_lora_grad_prequantized(const void* dy, tp_dtype dy_dtype, int64_t lddy, const int8_t* qa, int64_t ldqa,
                                    const float* sa, const float* t, const void* lora_b, tp_dtype b_dtype,
                                    int64_t ldb, float alpha, int a_flags, int64_t m, int64_t n, int64_t k, int64_t r,
                                    float* dt, float* da, int64_t ldda, float* db, int64_t lddb, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dy_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "dy_dtype %d is not TP_F32 or TP_BF16", (int)dy_dtype);
  if (!dtype_ok(b_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "b_dtype %d is not TP_F32 or TP_BF16", (int)b_dtype);
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  TP_TRY(check_sizes(m, n, k));
  TP_TRY(check_rank(r));
  if (m >= SIDE_MAX || n >= SIDE_MAX || k >= SIDE_MAX)
    return fail(TP_ERR_BAD_SHAPE, "m=%lld, n=%lld, k=%lld: below 2^26 each", (long long)m, (long long)n, (long long)k);
  const int64_t ys = dtype_size(dy_dtype), bs = dtype_size(b_dtype);
  Extent edy, eq, es, et, eb, edt, eda, edb, ew;
  TP_TRY(check_matrix("dy", dy, m, n * ys, lddy, ys, &edy));
  TP_TRY(check_matrix("qa", qa, m, k, ldqa, 1, &eq));
  TP_TRY(check_vector("sa", sa, m, &es));
  TP_TRY(check_matrix("t", t, m, 64 * 4, 64, 4, &et));
  TP_TRY(check_matrix("lora_b", lora_b, n, r * bs, ldb, bs, &eb));
  TP_TRY(check_matrix("dt", dt, m, 64 * 4, 64, 4, &edt));
  TP_TRY(check_matrix("da", da, r, k * 4, ldda, 4, &eda));
  TP_TRY(check_matrix("db", db, n, r * 4, lddb, 4, &edb, 4));
  TP_TRY(check_scratch("tp_lora_grad_workspace_size", workspace, workspace_bytes,
                       (int64_t)tp_lora_grad_workspace_size(m, n, k, r), &ew));
  const Extent* ins[] = {&edy, &eq, &es, &et, &eb};
  const Extent* outs[] = {&edt, &eda, &edb, &ew};
  for (int o = 0; o < 4; ++o) {
    for (const Extent* i : ins)
      if (overlaps(*outs[o], *i)) return fail(TP_ERR_BAD_ALIASING, "an output or the workspace overlaps an input");
    for (int p = 0; p < o; ++p)
      if (overlaps(*outs[o], *outs[p])) return fail(TP_ERR_BAD_ALIASING, "dt, da, db and the workspace must not overlap");
  }
  tp::SideGradArgs a{};
  a.dy = dy;
  a.dy_bf16 = dy_dtype == TP_BF16;
  a.lddy = lddy;
  a.qa = qa;
  a.ldqa = ldqa;
  a.sa = sa;
  a.t = t;
  a.b = lora_b;
  a.b_bf16 = b_dtype == TP_BF16;
  a.ldb = ldb;
  a.alpha = alpha;
  a.rotate = a_flags == TP_A_ROTATE;
  a.m = m;
  a.n = n;
  a.k = k;
  a.r = (int)r;
  a.dt = dt;
  a.da = da;
  a.ldda = ldda;
  a.db = db;
  a.lddb = lddb;
  a.ws = (float*)workspace;
  return hip_status(tp::launch_side_grad(a, stream), "side path gradient launch");
}

// ----------------------------------------------- norm and positions of q and k

namespace {

// A checked matrix: where its rows are.
struct MatRef {
  const void* p = nullptr;
  int dtype = 0;
  int64_t ld = 0;
  int64_t pitch = 0, row = 0;  // bytes
  Extent e;
};

tp_status check_ref(const char* name, const void* p, tp_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                    MatRef* r) {
  const int64_t es = dtype_size(dtype);
  TP_TRY(check_matrix(name, p, rows, cols * es, ld, es, &r->e));
  r->p = p;
  r->dtype = dtype;
  r->ld = ld;
  r->pitch = ld * es;
  r->row = cols * es;
  return TP_OK;
}

// Whether two matrices share bytes; column views of one buffer (equal pitches)
// do only where their columns do.
bool share(const MatRef& a, const MatRef& b) {
  if (!overlaps(a.e, b.e)) return false;
  if (a.pitch != b.pitch || a.pitch == 0) return true;
  const MatRef &lo = a.e.lo <= b.e.lo ? a : b, &hi = a.e.lo <= b.e.lo ? b : a;
  const int64_t delta = (int64_t)((hi.e.lo - lo.e.lo) % (uintptr_t)lo.pitch);
  return !(delta >= lo.row && delta + hi.row <= lo.pitch);
}

bool same_ref(const MatRef& a, const MatRef& b) { return a.p == b.p && a.dtype == b.dtype && a.ld == b.ld; }

// What forward and backward have in common.
tp_status check_rope(int64_t m, int64_t heads_q, int64_t heads_k, int64_t head_dim, const void* q_gamma,
                     const void* k_gamma, tp_dtype g_dtype, double eps, const int32_t* positions, int64_t ldpos,
                     int axes, const float* inv_freq, const uint8_t* pair_axis, int64_t pairs, int layout,
                     tp::RopeArgs* a, Extent* small /* [4] */) {
  if (m < 0 || m > INT_MAX) return fail(TP_ERR_BAD_SHAPE, "m=%lld", (long long)m);
  if (heads_q < 0 || heads_k < 0 || heads_q > tp::ROPE_MAX_HEADS || heads_k > tp::ROPE_MAX_HEADS ||
      heads_q + heads_k > tp::ROPE_MAX_HEADS)
    return fail(TP_ERR_BAD_SHAPE, "heads_q=%lld, heads_k=%lld: 0..%d together", (long long)heads_q, (long long)heads_k,
                tp::ROPE_MAX_HEADS);
  if (head_dim < 8 || head_dim % 8 != 0 || head_dim > tp::ROPE_MAX_DIM)
    return fail(TP_ERR_BAD_SHAPE, "head_dim=%lld: a multiple of 8 up to %d", (long long)head_dim, tp::ROPE_MAX_DIM);
  if (pairs < 0 || pairs % 4 != 0 || 2 * pairs > head_dim)
    return fail(TP_ERR_BAD_SHAPE, "pairs=%lld: a multiple of 4 up to head_dim / 2", (long long)pairs);
  if (layout != TP_ROPE_INTERLEAVED && layout != TP_ROPE_HALVES) return fail(TP_ERR_BAD_FLAGS, "layout=%d", layout);
  TP_TRY(check_eps(eps));
  TP_TRY(check_weight("q_gamma", q_gamma, g_dtype, head_dim, &small[0]));
  TP_TRY(check_weight("k_gamma", k_gamma, g_dtype, head_dim, &small[1]));
  small[2] = small[3] = Extent{};
  if (pairs > 0) {
    if (axes < 1 || axes > 4) return fail(TP_ERR_BAD_SHAPE, "axes=%d outside [1, 4]", axes);
    if (!pair_axis) return fail(TP_ERR_NULL_POINTER, "pair_axis is NULL");
    for (int64_t p = 0; p < pairs; ++p) {
      if (pair_axis[p] >= axes)
        return fail(TP_ERR_BAD_VALUE, "pair_axis[%lld]=%d, axes=%d", (long long)p, (int)pair_axis[p], axes);
      a->axis[p] = pair_axis[p];
    }
    TP_TRY(check_matrix("positions", positions, m, (int64_t)axes * 4, ldpos, 4, &small[2], 4));
    TP_TRY(check_vector("inv_freq", inv_freq, pairs, &small[3]));
  }
  a->m = m;
  a->heads_q = (int)heads_q;
  a->heads_k = (int)heads_k;
  a->head_dim = (int)head_dim;
  a->q_gamma = {q_gamma, q_gamma && g_dtype == TP_BF16};
  a->k_gamma = {k_gamma, k_gamma && g_dtype == TP_BF16};
  a->eps = eps;
  a->positions = positions;
  a->ldpos = ldpos;
  a->inv_freq = inv_freq;
  a->pairs = (int)pairs;
  a->halves = layout == TP_ROPE_HALVES;
  return TP_OK;
}

}  // namespace

tp_status tp_qk_norm_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, tp_dtype x_dtype, int64_t m,
                          int64_t heads_q, int64_t heads_k, int64_t head_dim, const void* q_gamma,
                          const void* k_gamma, tp_dtype g_dtype, double eps, const int32_t* positions, int64_t ldpos,
                          int axes, const float* inv_freq, const uint8_t* pair_axis, int64_t pairs, int layout,
                          void* q_out, int64_t ldqo, void* k_out, int64_t ldko, tp_dtype out_dtype,
                          hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (!dtype_ok(out_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "out_dtype %d is not TP_F32 or TP_BF16", (int)out_dtype);
  tp::RopeArgs a{};
  Extent small[4];
  TP_TRY(check_rope(m, heads_q, heads_k, head_dim, q_gamma, k_gamma, g_dtype, eps, positions, ldpos, axes, inv_freq,
                    pair_axis, pairs, layout, &a, small));
  MatRef in[2], out[2];
  TP_TRY(check_ref("q", q, x_dtype, m, heads_q * head_dim, ldq, &in[0]));
  TP_TRY(check_ref("k", k, x_dtype, m, heads_k * head_dim, ldk, &in[1]));
  TP_TRY(check_ref("q_out", q_out, out_dtype, m, heads_q * head_dim, ldqo, &out[0]));
  TP_TRY(check_ref("k_out", k_out, out_dtype, m, heads_k * head_dim, ldko, &out[1]));
  for (int o = 0; o < 2; ++o) {
    for (int i = 0; i < 2; ++i)
      if (share(out[o], in[i]) && !(o == i && same_ref(out[o], in[i])))
        return fail(TP_ERR_BAD_ALIASING, "%s overlaps an input without being its own", o ? "k_out" : "q_out");
    for (const Extent& e : small)
      if (overlaps(out[o].e, e)) return fail(TP_ERR_BAD_ALIASING, "an output overlaps a weight, positions or inv_freq");
  }
  if (share(out[0], out[1])) return fail(TP_ERR_BAD_ALIASING, "q_out and k_out overlap");
  if (m == 0 || heads_q + heads_k == 0) return ok();
  a.q = q;
  a.ldq = ldq;
  a.k = k;
  a.ldk = ldk;
  a.x_bf16 = x_dtype == TP_BF16;
  a.q_out = q_out;
  a.ldqo = ldqo;
  a.k_out = k_out;
  a.ldko = ldko;
  a.out_bf16 = out_dtype == TP_BF16;
  return hip_status(tp::launch_rope(a, stream), "rope launch");
}

size_t tp_qk_norm_rope_workspace_size(int64_t m, int64_t heads_q, int64_t heads_k, int64_t head_dim) {
  if (m <= 0 || m > INT_MAX || heads_q < 0 || heads_k < 0 || heads_q > tp::ROPE_MAX_HEADS ||
      heads_k > tp::ROPE_MAX_HEADS || heads_q + heads_k > tp::ROPE_MAX_HEADS || head_dim < 8 || head_dim % 8 != 0 ||
      head_dim > tp::ROPE_MAX_DIM)
    return 0;
  return (size_t)(tp::rope_partial_rows(m, (int)(heads_q + heads_k), (int)head_dim) * 2 * head_dim * 4);
}

tp_status tp_qk_norm_rope_backward(const void* dq_out, int64_t lddqo, const void* dk_out, int64_t lddko,
                                   tp_dtype dy_dtype, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                   tp_dtype x_dtype, int64_t m, int64_t heads_q, int64_t heads_k, int64_t head_dim,
                                   const void* q_gamma, const void* k_gamma, tp_dtype g_dtype, double eps,
                                   const int32_t* positions, int64_t ldpos, int axes, const float* inv_freq,
                                   const uint8_t* pair_axis, int64_t pairs, int layout, void* dq, int64_t lddq,
                                   void* dk, int64_t lddk, tp_dtype dx_dtype, float* dq_gamma, float* dk_gamma,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dy_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "dy_dtype %d is not TP_F32 or TP_BF16", (int)dy_dtype);
  if (!dtype_ok(dx_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "dx_dtype %d is not TP_F32 or TP_BF16", (int)dx_dtype);
  if ((q_gamma || k_gamma) && !dtype_ok(x_dtype))
    return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  tp::RopeArgs a{};
  Extent small[4];
  TP_TRY(check_rope(m, heads_q, heads_k, head_dim, q_gamma, k_gamma, g_dtype, eps, positions, ldpos, axes, inv_freq,
                    pair_axis, pairs, layout, &a, small));
  if ((dq_gamma && !q_gamma) || (dk_gamma && !k_gamma))
    return fail(TP_ERR_NULL_POINTER, "the gradient of a weight that is NULL");
  MatRef dy[2], in[2], out[2];
  TP_TRY(check_ref("dq_out", dq_out, dy_dtype, m, heads_q * head_dim, lddqo, &dy[0]));
  TP_TRY(check_ref("dk_out", dk_out, dy_dtype, m, heads_k * head_dim, lddko, &dy[1]));
  if (q_gamma) TP_TRY(check_ref("q", q, x_dtype, m, heads_q * head_dim, ldq, &in[0]));
  if (k_gamma) TP_TRY(check_ref("k", k, x_dtype, m, heads_k * head_dim, ldk, &in[1]));
  TP_TRY(check_ref("dq", dq, dx_dtype, m, heads_q * head_dim, lddq, &out[0]));
  TP_TRY(check_ref("dk", dk, dx_dtype, m, heads_k * head_dim, lddk, &out[1]));
  Extent edg[2] = {}, ew;
  if (dq_gamma) TP_TRY(check_vector("dq_gamma", dq_gamma, head_dim, &edg[0]));
  if (dk_gamma) TP_TRY(check_vector("dk_gamma", dk_gamma, head_dim, &edg[1]));
  const bool want = dq_gamma || dk_gamma;
  TP_TRY(check_scratch("tp_qk_norm_rope_workspace_size", workspace, workspace_bytes,
                       want ? (int64_t)tp_qk_norm_rope_workspace_size(m, heads_q, heads_k, head_dim) : 0, &ew));
  for (int o = 0; o < 2; ++o) {
    for (int i = 0; i < 2; ++i) {
      if (share(out[o], dy[i]) && !(o == i && same_ref(out[o], dy[i])))
        return fail(TP_ERR_BAD_ALIASING, "%s overlaps an output gradient without being its own", o ? "dk" : "dq");
      if (share(out[o], in[i]) && !(o == i && same_ref(out[o], in[i])))
        return fail(TP_ERR_BAD_ALIASING, "%s overlaps q or k without being its own", o ? "dk" : "dq");
    }
    for (const Extent& e : small)
      if (overlaps(out[o].e, e) || overlaps(edg[o], e) || overlaps(ew, e))
        return fail(TP_ERR_BAD_ALIASING, "an output or the workspace overlaps a weight, positions or inv_freq");
  }
  if (share(out[0], out[1])) return fail(TP_ERR_BAD_ALIASING, "dq and dk overlap");
  const Extent* mats[] = {&dy[0].e, &dy[1].e, &in[0].e, &in[1].e, &out[0].e, &out[1].e};
  for (const Extent* e : mats)
    if (overlaps(*e, edg[0]) || overlaps(*e, edg[1]) || overlaps(*e, ew))
      return fail(TP_ERR_BAD_ALIASING, "a weight's gradient or the workspace overlaps another operand");
  if (overlaps(edg[0], edg[1]) || overlaps(edg[0], ew) || overlaps(edg[1], ew))
    return fail(TP_ERR_BAD_ALIASING, "the weights' gradients and the workspace must not overlap");
  if ((m == 0 || heads_q + heads_k == 0) && !want) return ok();
  a.q = q;
  a.ldq = ldq;
  a.k = k;
  a.ldk = ldk;
  a.x_bf16 = (q_gamma || k_gamma) && x_dtype == TP_BF16;
  a.q_out = dq;
  a.ldqo = lddq;
  a.k_out = dk;
  a.ldko = lddk;
  a.out_bf16 = dx_dtype == TP_BF16;
  a.backward = 1;
  a.dq_out = dq_out;
  a.lddqo = lddqo;
  a.dk_out = dk_out;
  a.lddko = lddko;
  a.dy_bf16 = dy_dtype == TP_BF16;
  a.dq_gamma = dq_gamma;
  a.dk_gamma = dk_gamma;
  a.want_dgamma = want;
  a.part = (float*)workspace;
  return hip_status(tp::launch_rope(a, stream), "rope backward launch");
}

// --------------------------------------------- dropout and layer norm of rows

namespace {

// p in [0, 1] and the device memory of seed and offset (needed where something
// may drop; NULL where it is not used).
tp_status check_drop(double p, const uint64_t* rng, tp::DropArg* d, Extent* e) {
  *d = tp::DropArg{nullptr, 0, 1.f};
  *e = Extent{};
  if (!(p >= 0.0) || !(p <= 1.0)) return fail(TP_ERR_BAD_VALUE, "drop_p=%g is not within 0 .. 1", p);
  if (p == 0.0) return TP_OK;
  if (!rng) return fail(TP_ERR_NULL_POINTER, "rng is NULL (drop_p=%g)", p);
  if (((uintptr_t)rng & 7u) != 0) return fail(TP_ERR_MISALIGNED, "rng is not 8-byte aligned");
  e->lo = (uintptr_t)rng;
  e->hi = e->lo + 16;
  d->threshold = (uint32_t)nearbyint(p * 65536.0);
  d->scale = d->threshold < 65536u ? (float)(65536.0 / (65536.0 - (double)d->threshold)) : 0.f;
  d->rng = d->threshold > 0 ? rng : nullptr;  // (p below 2^-17 drops nothing)
  return TP_OK;
}

}  // namespace

tp_status tp_dropout(const void* x, tp_dtype x_dtype, int64_t ldx, const void* residual, int64_t ldr, double drop_p,
                     const uint64_t* rng, int64_t m, int64_t k, void* y, tp_dtype y_dtype, int64_t ldy,
                     hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (!dtype_ok(y_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "y_dtype %d is not TP_F32 or TP_BF16", (int)y_dtype);
  if (m < 0 || m > INT_MAX || k < 0 || k > INT_MAX)
    return fail(TP_ERR_BAD_SHAPE, "m=%lld, k=%lld", (long long)m, (long long)k);
  tp::DropoutArgs a{};
  Extent er, ex, es{}, ey;
  TP_TRY(check_drop(drop_p, rng, &a.drop, &er));
  const int64_t xs = dtype_size(x_dtype), ys = dtype_size(y_dtype);
  TP_TRY(check_matrix("x", x, m, k * xs, ldx, xs, &ex));
  if (residual) TP_TRY(check_matrix("residual", residual, m, k * ys, ldr, ys, &es));
  TP_TRY(check_matrix("y", y, m, k * ys, ldy, ys, &ey));
  if (overlaps(ey, er)) return fail(TP_ERR_BAD_ALIASING, "y overlaps rng");
  if (overlaps(ey, ex) && !same_buffer(y, y_dtype, ldy, x, x_dtype, ldx))
    return fail(TP_ERR_BAD_ALIASING, "y overlaps x without being the same buffer");
  if (overlaps(ey, es) && !same_buffer(y, y_dtype, ldy, residual, y_dtype, ldr))
    return fail(TP_ERR_BAD_ALIASING, "y overlaps residual without being the same buffer");
  if (m == 0 || k == 0) return ok();
  a.x = x;
  a.x_bf16 = x_dtype == TP_BF16;
  a.ldx = ldx;
  a.res = residual;
  a.ldr = ldr;
  a.m = m;
  a.k = k;
  a.y = y;
  a.y_bf16 = y_dtype == TP_BF16;
  a.ldy = ldy;
  return hip_status(tp::launch_dropout(a, stream), "dropout launch");
}

tp_status tp_layernorm_rotate(const void* x, tp_dtype x_dtype, int64_t ldx, const void* residual, int64_t ldr,
                              void* sum_out, int64_t ldsum, tp_dtype s_dtype, const void* gamma, const void* beta,
                              tp_dtype g_dtype, double eps, double drop_p, const uint64_t* rng, int a_flags, int64_t m,
                              int64_t k, int out_kind, void* y, int64_t ldy, float* scales, int64_t ldscales,
                              hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (out_kind != TP_NORM_OUT_I8 && out_kind != TP_NORM_OUT_BF16 && out_kind != TP_NORM_OUT_FP8)
    return fail(TP_ERR_BAD_FLAGS, "out_kind=%d", out_kind);
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  TP_TRY(check_sizes(m, 0, k));
  TP_TRY(check_norm_k(k));
  TP_TRY(check_eps(eps));
  const bool i8 = out_kind == TP_NORM_OUT_I8, bf16 = out_kind == TP_NORM_OUT_BF16;
  const int64_t xs = dtype_size(x_dtype), os = bf16 ? 2 : 1;
  tp::LayerNormArgs a{};
  Extent ex, er{}, esum{}, eg, eb, ey, esc{}, erng;
  TP_TRY(check_drop(drop_p, rng, &a.drop, &erng));
  TP_TRY(check_matrix("x", x, m, k * xs, ldx, xs, &ex));
  if (residual || sum_out) {
    if (!dtype_ok(s_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "s_dtype %d is not TP_F32 or TP_BF16", (int)s_dtype);
    const int64_t ss = dtype_size(s_dtype);
    if (!residual || !sum_out)
      return fail(TP_ERR_NULL_POINTER, "residual and sum_out are given together or not at all");
    TP_TRY(check_matrix("residual", residual, m, k * ss, ldr, ss, &er));
    TP_TRY(check_matrix("sum_out", sum_out, m, k * ss, ldsum, ss, &esum));
  } else if (drop_p != 0.0 && m > 0) {  // (no rows: empty tensors have no address)
    return fail(TP_ERR_NULL_POINTER, "drop_p=%g needs a residual and sum_out", drop_p);
  }
  TP_TRY(check_weight("gamma", gamma, g_dtype, k, &eg));
  TP_TRY(check_weight("beta", beta, g_dtype, k, &eb));
  TP_TRY(check_matrix("y", y, m, k * os, ldy, os, &ey));
  if (i8) TP_TRY(check_vector("scales", scales, m, &esc));
  if (out_kind == TP_NORM_OUT_FP8) TP_TRY(check_matrix("scales", scales, k / 128, m * 4, ldscales, 4, &esc, 4));
  const Extent* ins[] = {&ex, &er, &esum, &eg, &eb, &erng};
  for (const Extent* i : ins)
    if (overlaps(ey, *i) || overlaps(esc, *i))
      return fail(TP_ERR_BAD_ALIASING, "y and scales must not overlap x, residual, sum_out, gamma, beta or rng");
  if (overlaps(ey, esc)) return fail(TP_ERR_BAD_ALIASING, "y and scales overlap");
  if (overlaps(esum, eg) || overlaps(esum, eb) || overlaps(esum, erng))
    return fail(TP_ERR_BAD_ALIASING, "sum_out overlaps gamma, beta or rng");
  if (overlaps(esum, er) && !same_buffer(sum_out, s_dtype, ldsum, residual, s_dtype, ldr))
    return fail(TP_ERR_BAD_ALIASING, "sum_out overlaps residual without being the same buffer");
  if (overlaps(esum, ex) && !same_buffer(sum_out, s_dtype, ldsum, x, x_dtype, ldx))
    return fail(TP_ERR_BAD_ALIASING, "sum_out overlaps x without being the same buffer");
  if (m == 0) return ok();
  a.x = x;
  a.x_bf16 = x_dtype == TP_BF16;
  a.ldx = ldx;
  a.res = residual;
  a.ldr = ldr;
  a.sum = sum_out;
  a.ldsum = ldsum;
  a.s_bf16 = residual && s_dtype == TP_BF16;
  a.gamma = {gamma, gamma && g_dtype == TP_BF16};
  a.beta = {beta, beta && g_dtype == TP_BF16};
  a.eps = eps;
  a.rotate = a_flags == TP_A_ROTATE;
  a.m = m;
  a.groups = (int)(k / 256);
  a.out = out_kind;
  a.y = y;
  a.ldy = ldy;
  a.scales = bf16 ? nullptr : scales;
  a.ldscales = ldscales;
  return hip_status(tp::launch_layernorm(a, stream), "layer norm launch");
}

size_t tp_layernorm_backward_workspace_size(int64_t m, int64_t k) {
  if (m <= 0 || k <= 0 || k % 256 != 0 || m > INT_MAX || k / 256 > tp::NORM_MAX_GROUPS) return 0;
  return (size_t)tp::layernorm_bwd_workspace_bytes(m, (int)(k / 256));
}

tp_status tp_layernorm_rotate_backward(const void* dy, tp_dtype dy_dtype, int64_t lddy, int a_flags, const void* t,
                                       tp_dtype t_dtype, int64_t ldt, const void* gamma, tp_dtype g_dtype, double eps,
                                       const void* dsum, int64_t ldds, double drop_p, const uint64_t* rng, int64_t m,
                                       int64_t k, void* dx, tp_dtype dx_dtype, int64_t lddx, void* dbranch,
                                       int64_t lddb, float* dgamma, float* dbeta, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dy_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "dy_dtype %d is not TP_F32 or TP_BF16", (int)dy_dtype);
  if (!dtype_ok(t_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "t_dtype %d is not TP_F32 or TP_BF16", (int)t_dtype);
  if (!dtype_ok(dx_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "dx_dtype %d is not TP_F32 or TP_BF16", (int)dx_dtype);
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  TP_TRY(check_sizes(m, 0, k));
  TP_TRY(check_norm_k(k));
  TP_TRY(check_eps(eps));
  const int64_t gs = dtype_size(dy_dtype), ts = dtype_size(t_dtype), xs = dtype_size(dx_dtype);
  tp::LayerNormBwdArgs a{};
  Extent edy, et, eg, eds{}, edx, edb{}, edg{}, edbt{}, ew, erng;
  TP_TRY(check_drop(drop_p, rng, &a.drop, &erng));
  TP_TRY(check_matrix("dy", dy, m, k * gs, lddy, gs, &edy));
  TP_TRY(check_matrix("t", t, m, k * ts, ldt, ts, &et));
  TP_TRY(check_weight("gamma", gamma, g_dtype, k, &eg));
  if (dsum) TP_TRY(check_matrix("dsum", dsum, m, k * xs, ldds, xs, &eds));
  TP_TRY(check_matrix("dx", dx, m, k * xs, lddx, xs, &edx));
  if (dbranch) TP_TRY(check_matrix("dbranch", dbranch, m, k * xs, lddb, xs, &edb));
  if (dgamma) TP_TRY(check_vector("dgamma", dgamma, k, &edg));
  if (dbeta) TP_TRY(check_vector("dbeta", dbeta, k, &edbt));
  TP_TRY(check_scratch("tp_layernorm_backward_workspace_size", workspace, workspace_bytes,
                       dgamma || dbeta ? (int64_t)tp_layernorm_backward_workspace_size(m, k) : 0, &ew));
  const Extent* ins[] = {&edy, &et, &eg, &eds, &erng};
  const Extent* outs[] = {&edb, &edg, &edbt, &ew};  // apart from everything
  for (int o = 0; o < 4; ++o) {
    for (const Extent* i : ins)
      if (overlaps(*outs[o], *i))
        return fail(TP_ERR_BAD_ALIASING, "dbranch, dgamma, dbeta or the workspace overlaps an input");
    if (overlaps(*outs[o], edx))
      return fail(TP_ERR_BAD_ALIASING, "dbranch, dgamma, dbeta or the workspace overlaps dx");
    for (int p = 0; p < o; ++p)
      if (overlaps(*outs[o], *outs[p]))
        return fail(TP_ERR_BAD_ALIASING, "dbranch, dgamma, dbeta and the workspace must not overlap");
  }
  if (overlaps(edx, et) || overlaps(edx, eg) || overlaps(edx, erng))
    return fail(TP_ERR_BAD_ALIASING, "dx overlaps t, gamma or rng");
  if (overlaps(edx, eds) && !same_buffer(dx, dx_dtype, lddx, dsum, dx_dtype, ldds))
    return fail(TP_ERR_BAD_ALIASING, "dx overlaps dsum without being the same buffer");
  // (wide rows' sums read dy after dx is written)
  if (overlaps(edx, edy) && (dgamma || dbeta || !same_buffer(dx, dx_dtype, lddx, dy, dy_dtype, lddy)))
    return fail(TP_ERR_BAD_ALIASING, "dx overlaps dy without being the same buffer, or dgamma or dbeta is wanted");
  if (m == 0 && !dgamma && !dbeta) return ok();
  a.dy = dy;
  a.dy_bf16 = dy_dtype == TP_BF16;
  a.lddy = lddy;
  a.rotate = a_flags == TP_A_ROTATE;
  a.t = t;
  a.t_bf16 = t_dtype == TP_BF16;
  a.ldt = ldt;
  a.gamma = {gamma, gamma && g_dtype == TP_BF16};
  a.eps = eps;
  a.dsum = dsum;
  a.ldds = ldds;
  a.m = m;
  a.groups = (int)(k / 256);
  a.dx = dx;
  a.dx_bf16 = dx_dtype == TP_BF16;
  a.lddx = lddx;
  a.dbranch = dbranch;
  a.lddb = lddb;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.part = (float*)workspace;
  return hip_status(tp::launch_layernorm_bwd(a, stream), "layer norm backward launch");
}

// ------------------------------------- products in 8-bit floating point (e4m3)

namespace {

// Sizes of the block-scaled products: the kernels hold rows and columns in 32
// bits, and a launch counts its threads in 32 bits.
constexpr int64_t F8_MAX = (int64_t)1 << 26;
constexpr int64_t F8_MAX_PITCH = (int64_t)1 << 24;  // offsets within a tile of 256 rows are held in 32 bits
constexpr int64_t F8_MAX_QUANTIZED = (int64_t)1 << 34, F8_MAX_PRODUCT = (int64_t)1 << 36;  // elements

tp_status check_f8_sizes(int64_t m, int64_t n, int64_t most, const char* what) {
  if (m < 0 || n < 0 || m >= F8_MAX || n >= F8_MAX)
    return fail(TP_ERR_BAD_SHAPE, "%s: %lld, %lld: 0 .. 2^26 - 1 each", what, (long long)m, (long long)n);
  if (m * n > most)
    return fail(TP_ERR_BAD_SHAPE, "%s: %lld x %lld: at most %lld elements", what, (long long)m, (long long)n,
                (long long)most);
  return TP_OK;
}

}  // namespace

tp_status tp_quantize_fp8(const void* x, tp_dtype x_dtype, int64_t ldx, int64_t m, int64_t k, int a_flags,
                          int block_rows, uint8_t* q, int64_t ldq, float* scales, int64_t ldscales, uint8_t* qt,
                          int64_t ldqt, float* scales_t, int64_t ldscales_t, hipStream_t stream) {
  if (!dtype_ok(x_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "x_dtype %d is not TP_F32 or TP_BF16", (int)x_dtype);
  if (a_flags != TP_A_ROTATE && a_flags != TP_A_PREROTATED) return fail(TP_ERR_BAD_FLAGS, "a_flags=%d", a_flags);
  if (block_rows != 1 && block_rows != 128) return fail(TP_ERR_BAD_FLAGS, "block_rows=%d (1 or 128)", block_rows);
  TP_TRY(check_f8_sizes(m, k, F8_MAX_QUANTIZED, "m, k"));
  if (a_flags == TP_A_ROTATE && k % 256 != 0)
    return fail(TP_ERR_K_NOT_MULTIPLE_OF_256, "k=%lld is not a multiple of 256 (the rotation group)", (long long)k);
  if ((q == nullptr) != (scales == nullptr) || (qt == nullptr) != (scales_t == nullptr))
    return fail(TP_ERR_NULL_POINTER, "codes and their scales are given together or not at all");
  const int64_t xs = dtype_size(x_dtype), kp = round_up(k, 128), mp = round_up(m, 128);
  const bool blocks = block_rows == 128;
  Extent ex, eo[4] = {};
  TP_TRY(check_matrix("x", x, m, k * xs, ldx, xs, &ex));
  if (!q && !qt) return m == 0 || k == 0 ? ok() : fail(TP_ERR_NULL_POINTER, "q or qt (or both) is needed");
  if (m == 0 || k == 0) return ok();
  if (q) {
    TP_TRY(check_matrix("q", q, m, kp, ldq, 1, &eo[0]));
    TP_TRY(check_matrix("scales", scales, blocks ? mp / 128 : kp / 128, (blocks ? kp / 128 : m) * 4, ldscales, 4, &eo[1],
                        4));
  }
  if (qt) {
    TP_TRY(check_matrix("qt", qt, k, mp, ldqt, 1, &eo[2]));
    TP_TRY(check_matrix("scales_t", scales_t, blocks ? kp / 128 : mp / 128, (blocks ? mp / 128 : k) * 4, ldscales_t, 4,
                        &eo[3], 4));
  }
  for (int o = 0; o < 4; ++o) {
    if (overlaps(eo[o], ex)) return fail(TP_ERR_BAD_ALIASING, "codes or scales overlap x");
    for (int p = 0; p < o; ++p)
      if (overlaps(eo[o], eo[p])) return fail(TP_ERR_BAD_ALIASING, "codes and scales must not overlap");
  }
  tp::QuantFp8Args a{};
  a.x = x;
  a.x_bf16 = x_dtype == TP_BF16;
  a.ldx = ldx;
  a.m = m;
  a.k = k;
  a.rotate = a_flags == TP_A_ROTATE;
  a.blocks = blocks;
  a.q = q;
  a.ldq = ldq;
  a.s = scales;
  a.lds = ldscales;
  a.qt = qt;
  a.ldqt = ldqt;
  a.st = scales_t;
  a.ldst = ldscales_t;
  return hip_status(tp::launch_quantize_fp8(a, stream), "fp8 quantizer launch");
}

size_t tp_qgemm_fp8_workspace_size(int64_t m, int64_t n, int64_t k, tp_dtype c_dtype) {
  if (!dtype_ok(c_dtype) || m <= 0 || n <= 0 || k <= 0 || k % 128 != 0 || m >= F8_MAX || n >= F8_MAX || k >= F8_MAX_PITCH ||
      m * n > F8_MAX_PRODUCT)
    return 0;
  return (size_t)tp::qgemm_fp8_partial_bytes(m, n, k, c_dtype == TP_BF16);
}

tp_status tp_qgemm_fp8(const uint8_t* a, int64_t lda, const float* a_scales, int64_t ldsa, const uint8_t* b,
                       int64_t ldb, const float* b_scales, int64_t ldsb, int b_block_rows, int64_t m, int64_t n,
                       int64_t k, void* c, tp_dtype c_dtype, int64_t ldc, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  if (!dtype_ok(c_dtype)) return fail(TP_ERR_UNSUPPORTED_DTYPE, "c_dtype %d is not TP_F32 or TP_BF16", (int)c_dtype);
  if (b_block_rows != 1 && b_block_rows != 128) return fail(TP_ERR_BAD_FLAGS, "b_block_rows=%d (1 or 128)", b_block_rows);
  TP_TRY(check_f8_sizes(m, n, F8_MAX_PRODUCT, "m, n"));
  if (k <= 0 || k % 128 != 0 || k >= F8_MAX_PITCH)
    return fail(TP_ERR_BAD_SHAPE, "k=%lld: a positive multiple of 128 below 2^24", (long long)k);
  const int64_t cs = dtype_size(c_dtype), kb = k / 128;
  const bool rows = b_block_rows == 1;
  Extent e[4], ec, ew;
  TP_TRY(check_matrix("a", a, m, k, lda, 1, &e[0]));
  TP_TRY(check_matrix("a_scales", a_scales, kb, m * 4, ldsa, 4, &e[1], 4));
  TP_TRY(check_matrix("b", b, n, k, ldb, 1, &e[2]));
  if (lda >= F8_MAX_PITCH || ldb >= F8_MAX_PITCH)
    return fail(TP_ERR_BAD_LEADING_DIM, "lda=%lld, ldb=%lld: below 2^24", (long long)lda, (long long)ldb);
  TP_TRY(check_matrix("b_scales", b_scales, rows ? kb : (n + 127) / 128, (rows ? n : kb) * 4, ldsb, 4, &e[3], 4));
  TP_TRY(check_matrix("c", c, m, n * cs, ldc, cs, &ec, cs));
  TP_TRY(check_scratch("tp_qgemm_fp8_workspace_size", workspace, workspace_bytes,
                       (int64_t)tp_qgemm_fp8_workspace_size(m, n, k, c_dtype), &ew));
  for (int i = 0; i < 4; ++i)
    if (overlaps(ec, e[i]) || overlaps(ew, e[i])) return fail(TP_ERR_BAD_ALIASING, "c or the workspace overlaps an input");
  if (overlaps(ec, ew)) return fail(TP_ERR_BAD_ALIASING, "c and the workspace overlap");
  if (m == 0 || n == 0) return ok();
  tp::GemmFp8Args g{};
  g.a = a;
  g.lda = lda;
  g.sa = a_scales;
  g.ldsa = ldsa;
  g.b = b;
  g.ldb = ldb;
  g.sb = b_scales;
  g.ldsb = ldsb;
  g.b_rows = rows;
  g.m = m;
  g.n = n;
  g.k = k;
  g.c = c;
  g.c_bf16 = c_dtype == TP_BF16;
  g.ldc = ldc;
  g.part = (float*)workspace;
  return hip_status(tp::launch_qgemm_fp8(g, stream), "fp8 product launch");
}

}  // extern "C"
