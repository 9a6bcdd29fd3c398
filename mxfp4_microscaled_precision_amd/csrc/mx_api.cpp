// C ABI of the MXFP4 library (its MXFP8 comparator, the norm and the gradient
// clipping included): argument validation and launch dispatch.
// Every check runs on the host before anything is enqueued, so an invalid
// call launches nothing and writes nothing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <utility>

#include "../../include/mxfp4.h"
#include "mx_kernels.h"

namespace {

// HIP error behind the most recent MX_ERR_HIP returned on this thread.
thread_local hipError_t g_last_hip_error = hipSuccess;

mx_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MX_OK;
  g_last_hip_error = e;
  return MX_ERR_HIP;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_rotate(int32_t r) {
  return r == MX_ROT_NONE || r == MX_ROT_HADAMARD || r == MX_ROT_RAND_SIGN_HADAMARD ||
         r == MX_ROT_HADAMARD16;
}
bool valid_round(int32_t r) { return r == MX_ROUND_RNE || r == MX_ROUND_SR; }
bool valid_format(int32_t f) { return f == MX_FMT_FP4_E2M1 || f == MX_FMT_FP8_E4M3; }

// Code bytes per element, times two (E2M1: half a byte; E4M3: one byte).
int64_t code_bytes_x2(int32_t format) { return format == MX_FMT_FP8_E4M3 ? 2 : 1; }

// Reduction (K) and non-reduction (MN) extents of a quantized operand.
void operand_extents(const mx_qtensor *q, int64_t *mn, int64_t *k) {
  if (q->axis == 1) {
    *mn = q->rows;
    *k = q->cols;
  } else {
    *mn = q->cols;
    *k = q->rows;
  }
}

// Tiled-layout extents: MN up to a multiple of 256, K up to a multiple of 128
// (empty operands stay empty).
void padded_extents(int64_t rows, int64_t cols, int32_t axis, int64_t *mnp, int64_t *kp) {
  const int64_t mn = axis == 1 ? rows : cols;
  const int64_t k = axis == 1 ? cols : rows;
  const bool empty = rows == 0 || cols == 0;
  *mnp = empty ? 0 : (mn + 255) / 256 * 256;
  *kp = empty ? 0 : (k + 127) / 128 * 128;
}

// The GEMM addresses each operand's codes with 32-bit signed offsets (one
// 256-row block tile past the end must still be representable).
constexpr int64_t kMaxCodeBytes = (int64_t)1 << 30;

// Larger extents are unsupported: with at least 32 elements along the other
// axis their codes would pass the limit above anyway, and below it the
// product of two padded extents cannot overflow int64.
constexpr int64_t kMaxExtent = (int64_t)1 << 31;

bool extents_too_large(int64_t rows, int64_t cols) {
  return rows > kMaxExtent || cols > kMaxExtent;
}

// True when `rows` rows of `ld` elements of `elem_bytes` bytes each span more
// than 2^62 bytes, which no addressing in the kernels is built for
// (rows <= kMaxExtent).
bool span_too_large(int64_t rows, int64_t ld, int64_t elem_bytes) {
  return rows > 0 && ld > (((int64_t)1 << 62) / elem_bytes) / rows;
}

mx_status check_qtensor(const mx_qtensor *q) {
  if (q == nullptr) return MX_ERR_NULL;
  if (q->axis != 0 && q->axis != 1) return MX_ERR_ARG;
  if (q->block != 32) return MX_ERR_ARG;
  if (!valid_rotate(q->rotate) || !valid_round(q->round)) return MX_ERR_ARG;
  if (!valid_format(q->format)) return MX_ERR_ARG;
  if (q->format == MX_FMT_FP8_E4M3 && q->round != MX_ROUND_RNE) return MX_ERR_ARG;
  if (q->rows < 0 || q->cols < 0) return MX_ERR_SHAPE;
  const int64_t k = q->axis == 1 ? q->cols : q->rows;
  if (k % 32 != 0) return MX_ERR_SHAPE;
  if (q->rows > 0 && q->cols > 0) {
    if (q->codes == nullptr || q->scales == nullptr) return MX_ERR_NULL;
    if (!aligned(q->codes, 16) || !aligned(q->scales, 4)) return MX_ERR_ALIGN;
    if (extents_too_large(q->rows, q->cols)) return MX_ERR_UNSUPPORTED;
    int64_t mnp, kp;
    padded_extents(q->rows, q->cols, q->axis, &mnp, &kp);
    if (mnp * kp * code_bytes_x2(q->format) / 2 >= kMaxCodeBytes) return MX_ERR_UNSUPPORTED;
  }
  return MX_OK;
}

void fill_desc(mx_qtensor *d, void *codes, void *scales, int64_t rows, int64_t cols,
               int32_t axis, int32_t block, int32_t rotate, int32_t round, uint64_t seed,
               int32_t format) {
  if (d == nullptr) return;
  d->codes = codes;
  d->scales = scales;
  d->rows = rows;
  d->cols = cols;
  d->axis = axis;
  d->block = block;
  d->rotate = rotate;
  d->round = round;
  d->seed = seed;
  d->format = format;
}

// Validation shared by the single-orientation quantize calls.
mx_status check_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld,
                         int32_t axis, int32_t block, int32_t rotate, int32_t round,
                         const void *codes, const void *scales, int32_t format) {
  if (axis != 0 && axis != 1) return MX_ERR_ARG;
  if (block != 32) return MX_ERR_ARG;
  if (!valid_rotate(rotate) || !valid_round(round)) return MX_ERR_ARG;
  if (rows < 0 || cols < 0) return MX_ERR_SHAPE;
  const int64_t k = axis == 1 ? cols : rows;
  if (k % 32 != 0) return MX_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MX_OK;
  if (x_bf16 == nullptr || codes == nullptr || scales == nullptr) return MX_ERR_NULL;
  if (ld < cols) return MX_ERR_SHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return MX_ERR_ALIGN;
  if (extents_too_large(rows, cols) || span_too_large(rows, ld, 2)) return MX_ERR_UNSUPPORTED;
  int64_t mnp, kp;
  padded_extents(rows, cols, axis, &mnp, &kp);
  if (mnp * kp * code_bytes_x2(format) / 2 >= kMaxCodeBytes) return MX_ERR_UNSUPPORTED;
  if (axis == 1) {
    if (ld % 8 != 0 || !aligned(x_bf16, 16)) return MX_ERR_ALIGN;
  } else {
    if (!aligned(x_bf16, 2)) return MX_ERR_ALIGN;
  }
  return MX_OK;
}

mx_status sizes(int64_t rows, int64_t cols, int32_t axis, int32_t block, int32_t format,
                size_t *codes_bytes, size_t *scales_bytes) {
  if (codes_bytes == nullptr || scales_bytes == nullptr) return MX_ERR_NULL;
  if (axis != 0 && axis != 1) return MX_ERR_ARG;
  if (block != 32) return MX_ERR_ARG;
  if (rows < 0 || cols < 0) return MX_ERR_SHAPE;
  const int64_t k = axis == 1 ? cols : rows;
  if (k % 32 != 0) return MX_ERR_SHAPE;
  if (rows > 0 && cols > 0 && extents_too_large(rows, cols)) return MX_ERR_UNSUPPORTED;
  int64_t mnp, kp;
  padded_extents(rows, cols, axis, &mnp, &kp);
  *codes_bytes = (size_t)(mnp * kp * code_bytes_x2(format) / 2);
  *scales_bytes = (size_t)mnp * (size_t)kp / 32;
  return MX_OK;
}

mx_status quantize_any(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld, int32_t axis,
                       int32_t block, int32_t rotate, int32_t round, uint64_t seed, void *codes,
                       void *scales, mx_qtensor *out_desc, void *stream, int32_t format) {
  const mx_status st =
      check_quantize(x_bf16, rows, cols, ld, axis, block, rotate, round, codes, scales, format);
  if (st != MX_OK) return st;
  fill_desc(out_desc, codes, scales, rows, cols, axis, block, rotate, round, seed, format);
  if (rows == 0 || cols == 0) return MX_OK;
  mx::QuantArgs a;
  a.x = static_cast<const uint16_t *>(x_bf16);
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.axis = axis;
  a.rotate = rotate;
  a.round = round;
  a.seed_lo = (uint32_t)(seed & 0xFFFFFFFFull);
  a.seed_hi = (uint32_t)(seed >> 32);
  a.codes = static_cast<uint8_t *>(codes);
  a.scales = static_cast<uint8_t *>(scales);
  a.rb = 0;
  a.fmt = format == MX_FMT_FP8_E4M3 ? 1 : 0;
  return hip_status(mx::quantize_launch(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

mx_status mx_quantize_sizes(int64_t rows, int64_t cols, int32_t axis, int32_t block,
                            size_t *codes_bytes, size_t *scales_bytes) {
  return sizes(rows, cols, axis, block, MX_FMT_FP4_E2M1, codes_bytes, scales_bytes);
}

mx_status mx_quantize_fp8_sizes(int64_t rows, int64_t cols, int32_t axis, int32_t block,
                                size_t *codes_bytes, size_t *scales_bytes) {
  return sizes(rows, cols, axis, block, MX_FMT_FP8_E4M3, codes_bytes, scales_bytes);
}

mx_status mx_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld, int32_t axis,
                      int32_t block, int32_t rotate, int32_t round, uint64_t seed, void *codes,
                      void *scales, mx_qtensor *out_desc, void *stream) {
  return quantize_any(x_bf16, rows, cols, ld, axis, block, rotate, round, seed, codes, scales,
                      out_desc, stream, MX_FMT_FP4_E2M1);
}

mx_status mx_quantize_fp8(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld,
                          int32_t axis, int32_t block, int32_t rotate, uint64_t seed,
                          void *codes, void *scales, mx_qtensor *out_desc, void *stream) {
  return quantize_any(x_bf16, rows, cols, ld, axis, block, rotate, MX_ROUND_RNE, seed, codes,
                      scales, out_desc, stream, MX_FMT_FP8_E4M3);
}

mx_status mx_quantize_pair(const void *xa_bf16, int64_t rows_a, int64_t lda,
                           const void *xb_bf16, int64_t rows_b, int64_t ldb, int64_t cols,
                           int32_t block, int32_t rotate, int32_t round, uint64_t seed_a,
                           uint64_t seed_b, void *codes_a, void *scales_a, void *codes_b,
                           void *scales_b, mx_qtensor *desc_a, mx_qtensor *desc_b,
                           void *stream) {
  mx_status st = check_quantize(xa_bf16, rows_a, cols, lda, 1, block, rotate, round, codes_a,
                                scales_a, MX_FMT_FP4_E2M1);
  if (st != MX_OK) return st;
  st = check_quantize(xb_bf16, rows_b, cols, ldb, 1, block, rotate, round, codes_b, scales_b,
                      MX_FMT_FP4_E2M1);
  if (st != MX_OK) return st;
  fill_desc(desc_a, codes_a, scales_a, rows_a, cols, 1, block, rotate, round, seed_a,
            MX_FMT_FP4_E2M1);
  fill_desc(desc_b, codes_b, scales_b, rows_b, cols, 1, block, rotate, round, seed_b,
            MX_FMT_FP4_E2M1);
  const bool live_a = rows_a > 0 && cols > 0, live_b = rows_b > 0 && cols > 0;
  if (!live_a && !live_b) return MX_OK;
  mx::QuantArgs q[2];
  const void *xs[2] = {xa_bf16, xb_bf16};
  const int64_t rs[2] = {rows_a, rows_b}, lds[2] = {lda, ldb};
  const uint64_t seeds[2] = {seed_a, seed_b};
  void *cs[2] = {codes_a, codes_b}, *ss[2] = {scales_a, scales_b};
  for (int i = 0; i < 2; ++i) {
    q[i].x = static_cast<const uint16_t *>(xs[i]);
    q[i].rows = rs[i];
    q[i].cols = cols;
    q[i].ld = lds[i];
    q[i].axis = 1;
    q[i].rotate = rotate;
    q[i].round = round;
    q[i].seed_lo = (uint32_t)(seeds[i] & 0xFFFFFFFFull);
    q[i].seed_hi = (uint32_t)(seeds[i] >> 32);
    q[i].codes = static_cast<uint8_t *>(cs[i]);
    q[i].scales = static_cast<uint8_t *>(ss[i]);
    q[i].rb = 0;
    q[i].fmt = 0;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!live_b) return hip_status(mx::quantize_launch(q[0], s));
  if (!live_a) return hip_status(mx::quantize_launch(q[1], s));
  return hip_status(mx::quantize_pair_launch(q[0], q[1], s));
}

mx_status mx_quantize_dual(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld,
                           int32_t block, int32_t rotate, int32_t round, uint64_t seed1,
                           uint64_t seed0, void *codes1, void *scales1, void *codes0,
                           void *scales0, mx_qtensor *desc1, mx_qtensor *desc0, void *stream) {
  if (block != 32) return MX_ERR_ARG;
  if (!valid_rotate(rotate) || !valid_round(round)) return MX_ERR_ARG;
  if (rows < 0 || cols < 0) return MX_ERR_SHAPE;
  if (rows % 32 != 0 || cols % 32 != 0) return MX_ERR_SHAPE;
  const bool empty = rows == 0 || cols == 0;
  if (!empty) {
    if (x_bf16 == nullptr || codes1 == nullptr || scales1 == nullptr || codes0 == nullptr ||
        scales0 == nullptr)
      return MX_ERR_NULL;
    if (ld < cols) return MX_ERR_SHAPE;
    if (ld % 8 != 0 || !aligned(x_bf16, 16)) return MX_ERR_ALIGN;
    if (!aligned(codes1, 16) || !aligned(scales1, 4) || !aligned(codes0, 16) ||
        !aligned(scales0, 4))
      return MX_ERR_ALIGN;
    if (extents_too_large(rows, cols) || span_too_large(rows, ld, 2)) return MX_ERR_UNSUPPORTED;
    for (int axis = 0; axis < 2; ++axis) {
      int64_t mnp, kp;
      padded_extents(rows, cols, axis, &mnp, &kp);
      if (mnp * kp / 2 >= kMaxCodeBytes) return MX_ERR_UNSUPPORTED;
    }
  }
  fill_desc(desc0, codes0, scales0, rows, cols, 0, block, rotate, round, seed0, MX_FMT_FP4_E2M1);
  fill_desc(desc1, codes1, scales1, rows, cols, 1, block, rotate, round, seed1, MX_FMT_FP4_E2M1);
  if (empty) return MX_OK;

  mx::DualArgs a;
  a.x = static_cast<const uint16_t *>(x_bf16);
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.rotate = rotate;
  a.round = round;
  a.seed1_lo = (uint32_t)(seed1 & 0xFFFFFFFFull);
  a.seed1_hi = (uint32_t)(seed1 >> 32);
  a.seed0_lo = (uint32_t)(seed0 & 0xFFFFFFFFull);
  a.seed0_hi = (uint32_t)(seed0 >> 32);
  a.codes1 = static_cast<uint8_t *>(codes1);
  a.scales1 = static_cast<uint8_t *>(scales1);
  a.codes0 = static_cast<uint8_t *>(codes0);
  a.scales0 = static_cast<uint8_t *>(scales0);
  return hip_status(mx::quantize_dual_launch(a, static_cast<hipStream_t>(stream)));
}

namespace {

// mx_linear's checks of one (A, B, C) entry; fills the GEMM's extents and the
// entry's pointers. *empty is set when M or N is 0 (nothing to launch).
mx_status linear_entry(int32_t op, const mx_qtensor *A, const mx_qtensor *B, void *C, int64_t ldc,
                       int32_t out_dtype, mx::GemmArgs *g, bool *empty) {
  if (op != MX_OP_FPROP && op != MX_OP_DGRAD && op != MX_OP_WGRAD) return MX_ERR_ARG;
  if (out_dtype != MX_OUT_F32 && out_dtype != MX_OUT_BF16) return MX_ERR_ARG;
  mx_status st = check_qtensor(A);
  if (st != MX_OK) return st;
  st = check_qtensor(B);
  if (st != MX_OK) return st;
  // Which axis each operand must be quantized along, per op.
  static const int32_t need_axis[3][2] = {{1, 1}, {1, 0}, {0, 0}};
  if (A->axis != need_axis[op][0] || B->axis != need_axis[op][1]) return MX_ERR_ARG;
  if (A->rotate != B->rotate || A->format != B->format) return MX_ERR_MISMATCH;
  if (A->rotate == MX_ROT_RAND_SIGN_HADAMARD &&
      (uint32_t)(A->seed & 0xFFFFFFFFull) != (uint32_t)(B->seed & 0xFFFFFFFFull))
    return MX_ERR_MISMATCH;
  int64_t M, Ka, N, Kb;
  operand_extents(A, &M, &Ka);
  operand_extents(B, &N, &Kb);
  if (Ka != Kb) return MX_ERR_SHAPE;
  if (ldc < N) return MX_ERR_SHAPE;
  *empty = M == 0 || N == 0;
  if (!*empty) {
    if (C == nullptr) return MX_ERR_NULL;
    if (!aligned(C, out_dtype == MX_OUT_F32 ? 4 : 2)) return MX_ERR_ALIGN;
    if (span_too_large(M, ldc, out_dtype == MX_OUT_F32 ? 4 : 2)) return MX_ERR_UNSUPPORTED;
  }
  g->a_codes = static_cast<const uint8_t *>(A->codes);
  g->a_scales = static_cast<const uint8_t *>(A->scales);
  g->b_codes = static_cast<const uint8_t *>(B->codes);
  g->b_scales = static_cast<const uint8_t *>(B->scales);
  g->c = C;
  g->M = M;
  g->N = N;
  g->K = Ka;
  g->ldc = ldc;
  g->out_bf16 = out_dtype == MX_OUT_BF16 ? 1 : 0;
  return MX_OK;
}

}  // namespace

mx_status mx_linear(int32_t op, const mx_qtensor *A, const mx_qtensor *B, void *C, int64_t ldc,
                    int32_t out_dtype, void *stream) {
  mx::GemmArgs g;
  bool empty = false;
  const mx_status st = linear_entry(op, A, B, C, ldc, out_dtype, &g, &empty);
  if (st != MX_OK || empty) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return hip_status(A->format == MX_FMT_FP8_E4M3 ? mx::gemm_e4m3_launch(g, s)
                                                 : mx::gemm_launch(g, s));
}

mx_status mx_linear_batched(int32_t op, int32_t count, const mx_qtensor *A, const mx_qtensor *B,
                            void *const *C, int64_t ldc, int32_t out_dtype, void *stream) {
  if (count < 1 || count > mx::kMaxGemmBatch) return MX_ERR_ARG;
  if (A == nullptr || B == nullptr || C == nullptr) return MX_ERR_NULL;
  mx::GemmArgs g;
  bool empty = false;
  for (int32_t i = 0; i < count; ++i) {
    if (A[i].rows != A[0].rows || A[i].cols != A[0].cols || A[i].axis != A[0].axis ||
        B[i].rows != B[0].rows || B[i].cols != B[0].cols || B[i].axis != B[0].axis)
      return MX_ERR_SHAPE;
    mx::GemmArgs gi;
    const mx_status st = linear_entry(op, &A[i], &B[i], C[i], ldc, out_dtype, &gi, &empty);
    if (st != MX_OK) return st;
    if (A[i].format != MX_FMT_FP4_E2M1) return MX_ERR_UNSUPPORTED;
    if (i == 0)
      g = gi;
    else
      g.more[i - 1] = mx::GemmEntry{gi.a_codes, gi.a_scales, gi.b_codes, gi.b_scales, gi.c};
  }
  if (empty) return MX_OK;
  g.batch = count;
  return hip_status(mx::gemm_launch(g, static_cast<hipStream_t>(stream)));
}

mx_status mx_dequantize(const mx_qtensor *q, float *out, int64_t ld, void *stream) {
  const mx_status st = check_qtensor(q);
  if (st != MX_OK) return st;
  if (ld < q->cols) return MX_ERR_SHAPE;
  if (q->rows == 0 || q->cols == 0) return MX_OK;
  if (out == nullptr) return MX_ERR_NULL;
  if (!aligned(out, 4)) return MX_ERR_ALIGN;
  if (span_too_large(q->rows, ld, 4)) return MX_ERR_UNSUPPORTED;
  mx::DequantArgs a;
  a.codes = static_cast<const uint8_t *>(q->codes);
  a.scales = static_cast<const uint8_t *>(q->scales);
  operand_extents(q, &a.mn, &a.k);
  padded_extents(q->rows, q->cols, q->axis, &a.mnp, &a.kp);
  a.axis = q->axis;
  a.fmt = q->format == MX_FMT_FP8_E4M3 ? 1 : 0;
  a.out = out;
  a.ld = ld;
  return hip_status(mx::dequantize_launch(a, static_cast<hipStream_t>(stream)));
}

namespace {

// (static: within extern "C" an unnamed namespace alone does not hide a name)
static bool valid_dtype(int32_t t) { return t == MX_OUT_F32 || t == MX_OUT_BF16; }
static int64_t dtype_size(int32_t t) { return t == MX_OUT_F32 ? 4 : 2; }

// A [rows, cols] matrix that the norm kernels read or write in 16-byte units.
static mx_status check_rows(const void *p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
  if (p == nullptr) return MX_ERR_NULL;
  if (ld < cols) return MX_ERR_SHAPE;
  if (!aligned(p, 16) || ld % (16 / dtype_size(dtype)) != 0) return MX_ERR_ALIGN;
  if (span_too_large(rows, ld, dtype_size(dtype))) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

}  // namespace

mx_status mx_rmsnorm_quantize(const mx_norm *n, int32_t format, int32_t block, int32_t rotate,
                              int32_t round, uint64_t seed1, uint64_t seed0, void *codes1,
                              void *scales1, void *codes0, void *scales0, mx_qtensor *desc1,
                              mx_qtensor *desc0, void *stream) {
  if (n == nullptr) return MX_ERR_NULL;
  if (block != 32) return MX_ERR_ARG;
  if (!valid_rotate(rotate) || !valid_round(round) || !valid_format(format)) return MX_ERR_ARG;
  if (format == MX_FMT_FP8_E4M3 && round != MX_ROUND_RNE) return MX_ERR_ARG;
  if (!valid_dtype(n->dtype) || !valid_dtype(n->weight_dtype)) return MX_ERR_ARG;
  if (!(n->eps >= 0.0) || std::isinf(n->eps)) return MX_ERR_ARG;
  const int64_t rows = n->rows, cols = n->cols;
  if (rows < 0 || cols < 0) return MX_ERR_SHAPE;
  const bool dual = codes0 != nullptr || scales0 != nullptr;
  if (cols % 32 != 0 || (dual && rows % 32 != 0)) return MX_ERR_SHAPE;
  const bool empty = rows == 0 || cols == 0;
  if (!empty) {
    if (n->weight == nullptr || n->rstd == nullptr || codes1 == nullptr || scales1 == nullptr ||
        (dual && (codes0 == nullptr || scales0 == nullptr)))
      return MX_ERR_NULL;
    if (extents_too_large(rows, cols)) return MX_ERR_UNSUPPORTED;
    mx_status st = check_rows(n->x, rows, cols, n->ldx, n->dtype);
    if (st != MX_OK) return st;
    if (n->residual != nullptr) {
      st = check_rows(n->residual, rows, cols, n->ldr, n->dtype);
      if (st != MX_OK) return st;
      st = check_rows(n->h, rows, cols, n->ldh, n->dtype);
      if (st != MX_OK) return st;
      if ((n->h == n->x && n->ldh != n->ldx) || (n->h == n->residual && n->ldh != n->ldr))
        return MX_ERR_SHAPE;
    }
    if (!aligned(n->weight, 16) || !aligned(n->rstd, 4) || !aligned(codes1, 16) ||
        !aligned(scales1, 4) || (dual && (!aligned(codes0, 16) || !aligned(scales0, 4))))
      return MX_ERR_ALIGN;
    for (int axis = dual ? 0 : 1; axis < 2; ++axis) {
      int64_t mnp, kp;
      padded_extents(rows, cols, axis, &mnp, &kp);
      if (mnp * kp * code_bytes_x2(format) / 2 >= kMaxCodeBytes) return MX_ERR_UNSUPPORTED;
    }
  }
  fill_desc(desc1, codes1, scales1, rows, cols, 1, block, rotate, round, seed1, format);
  if (dual) fill_desc(desc0, codes0, scales0, rows, cols, 0, block, rotate, round, seed0, format);
  if (empty) return MX_OK;

  mx::NormArgs a;
  a.x = n->x;
  a.residual = n->residual;
  a.weight = n->weight;
  a.h = n->residual != nullptr ? n->h : const_cast<void *>(n->x);   // never written without one
  a.rstd = n->rstd;
  a.rows = rows;
  a.cols = cols;
  a.ldx = n->ldx;
  a.ldr = n->ldr;
  a.ldh = n->residual != nullptr ? n->ldh : n->ldx;
  a.f32 = n->dtype == MX_OUT_F32 ? 1 : 0;
  a.wf32 = n->weight_dtype == MX_OUT_F32 ? 1 : 0;
  a.eps = n->eps;
  a.inv_cols = 1.0 / (double)cols;
  a.rotate = rotate;
  a.round = round;
  a.fmt = format == MX_FMT_FP8_E4M3 ? 1 : 0;
  a.seed1_lo = (uint32_t)(seed1 & 0xFFFFFFFFull);
  a.seed1_hi = (uint32_t)(seed1 >> 32);
  a.seed0_lo = (uint32_t)(seed0 & 0xFFFFFFFFull);
  a.seed0_hi = (uint32_t)(seed0 >> 32);
  a.codes1 = static_cast<uint8_t *>(codes1);
  a.scales1 = static_cast<uint8_t *>(scales1);
  a.codes0 = static_cast<uint8_t *>(codes0);
  a.scales0 = static_cast<uint8_t *>(scales0);
  return hip_status(mx::norm_launch(a, static_cast<hipStream_t>(stream)));
}

mx_status mx_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t *bytes) {
  if (bytes == nullptr) return MX_ERR_NULL;
  if (rows < 0 || cols < 0) return MX_ERR_SHAPE;
  if (extents_too_large(rows, cols)) return MX_ERR_UNSUPPORTED;
  *bytes = mx::norm_grad_few(rows, cols)
               ? 0
               : (size_t)mx::norm_grad_groups(rows, cols) * (size_t)cols * sizeof(float);
  return MX_OK;
}

mx_status mx_rmsnorm_backward(const mx_norm_grad *g, void *workspace, size_t workspace_bytes,
                              void *stream) {
  if (g == nullptr) return MX_ERR_NULL;
  if (!valid_dtype(g->dtype) || !valid_dtype(g->weight_dtype)) return MX_ERR_ARG;
  const int64_t rows = g->rows, cols = g->cols;
  size_t need = 0;
  mx_status st = mx_rmsnorm_backward_workspace(rows, cols, &need);
  if (st != MX_OK) return st;
  if (cols % 8 != 0) return MX_ERR_SHAPE;
  if (cols == 0) return MX_OK;
  if (g->dweight == nullptr) return MX_ERR_NULL;
  if (!aligned(g->dweight, 16)) return MX_ERR_ALIGN;
  if (rows > 0) {
    if (g->rstd == nullptr || g->weight == nullptr || (need > 0 && workspace == nullptr))
      return MX_ERR_NULL;
    const void *m[4] = {g->dy, g->h, g->dh, g->dres};
    const int64_t ld[4] = {g->lddy, g->ldh, g->lddh, g->ldres};
    for (int i = 0; i < (g->dres != nullptr ? 4 : 3); ++i) {
      st = check_rows(m[i], rows, cols, ld[i], g->dtype);
      if (st != MX_OK) return st;
    }
    if (g->dh == g->h) return MX_ERR_ARG;
    if ((g->dh == g->dy && g->lddh != g->lddy) || (g->dh == g->dres && g->lddh != g->ldres) ||
        workspace_bytes < need)
      return MX_ERR_SHAPE;
    if (!aligned(g->rstd, 4) || !aligned(g->weight, 16) || !aligned(workspace, 16))
      return MX_ERR_ALIGN;
  }
  mx::NormGradArgs a;
  a.dy = g->dy;
  a.h = g->h;
  a.dres = g->dres;
  a.rstd = g->rstd;
  a.weight = g->weight;
  a.dh = g->dh;
  a.dweight = g->dweight;
  a.partial = static_cast<float *>(workspace);
  a.rows = rows;
  a.cols = cols;
  a.lddy = g->lddy;
  a.ldh = g->ldh;
  a.ldres = g->ldres;
  a.lddh = g->lddh;
  a.f32 = g->dtype == MX_OUT_F32 ? 1 : 0;
  a.wf32 = g->weight_dtype == MX_OUT_F32 ? 1 : 0;
  return hip_status(mx::norm_grad_launch(a, static_cast<hipStream_t>(stream)));
}

namespace {

// A set's table: the tensors, the chunks, then the indices of the tensors that
// are not empty, those without gaps by address and then those with gaps by
// address (host only, for the overlap checks).
struct GradLayout {
  int64_t chunks, chunk, gapless, gapped;
  size_t chunks_at, order_at, bytes;
};

static bool grad_empty(const mx_grad &g) { return g.rows == 0 || g.cols == 0; }
static bool grad_gapless(const mx_grad &g) { return g.rows <= 1 || g.ld == g.cols; }
static int64_t grad_bytes(const mx_grad &g) { return g.rows * g.cols * dtype_size(g.dtype); }
static uintptr_t address(const mx_grad &g) { return reinterpret_cast<uintptr_t>(g.data); }

// A tensor's memory: count runs of `width` bytes, `pitch` apart (one run where
// there are no gaps).
struct GradRuns {
  uintptr_t start;
  int64_t count, width, pitch;
  uintptr_t end() const { return start + (uintptr_t)((count - 1) * pitch + width); }
};

static GradRuns grad_runs(const mx_grad &g) {
  if (grad_gapless(g)) return {address(g), 1, grad_bytes(g), grad_bytes(g)};
  const int64_t size = dtype_size(g.dtype);
  return {address(g), g.rows, g.cols * size, g.ld * size};
}

// Whether two tensors that are not empty share a byte. Run i of one and run j of
// the other with the same pitch lie d + (j - i) pitch apart, so the smallest
// j - i that ends past the other's start decides; with unequal pitches that is
// asked for each run of the tensor with fewer.
static bool grads_overlap(const mx_grad &p, const mx_grad &q) {
  GradRuns a = grad_runs(p), b = grad_runs(q);
  if (a.end() <= b.start || b.end() <= a.start) return false;
  if (a.count > b.count) std::swap(a, b);
  auto meet = [&b](uintptr_t start, int64_t count, int64_t width) {   // runs of b's pitch
    const int64_t d = (int64_t)(b.start - start);
    const int64_t past = -b.width - d;                  // of k pitches: strictly more than this
    int64_t k = past / b.pitch + (past % b.pitch < 0 ? 0 : 1);
    k = std::max(k, -(count - 1));
    return k <= b.count - 1 && d + k * b.pitch < width;
  };
  if (a.count == 1 || a.pitch == b.pitch) return meet(a.start, a.count, a.width);
  for (int64_t i = 0; i < a.count; ++i)
    if (meet(a.start + (uintptr_t)(i * a.pitch), 1, a.width)) return true;
  return false;
}

// Tensors by address.
struct GradOrder {
  const mx_grad *grads;
  const uint32_t *index;
  int64_t n;
};

// Whether a tensor of y starts within the span of one of x and shares memory
// with it, unless it is the same one at the same place of its set.
static bool any_clash(const GradOrder &x, const GradOrder &y) {
  const uint32_t *const end = y.index + y.n;
  for (int64_t i = 0; i < x.n && y.n > 0; ++i) {
    const mx_grad &p = x.grads[x.index[i]];
    const uintptr_t past = grad_runs(p).end();
    const uint32_t *j =
        std::lower_bound(y.index, end, address(p),
                         [&](uint32_t e, uintptr_t at) { return address(y.grads[e]) < at; });
    for (; j != end && address(y.grads[*j]) < past; ++j) {
      const mx_grad &q = y.grads[*j];
      const bool same = x.index[i] == *j && p.data == q.data &&
                        grad_runs(p).count == grad_runs(q).count &&
                        grad_runs(p).pitch == grad_runs(q).pitch;
      if (!same && grads_overlap(p, q)) return true;
    }
  }
  return false;
}

static mx_status grad_layout(int32_t count, const mx_grad *grads, GradLayout *l) {
  if (count < 0) return MX_ERR_ARG;
  if (count > 0 && grads == nullptr) return MX_ERR_NULL;
  int64_t total = 0;
  l->gapless = l->gapped = 0;
  for (int32_t i = 0; i < count; ++i) {
    const mx_grad &g = grads[i];
    if (!valid_dtype(g.dtype)) return MX_ERR_ARG;
    if (g.rows < 0 || g.cols < 0) return MX_ERR_SHAPE;
    if (grad_empty(g)) continue;
    if (g.data == nullptr) return MX_ERR_NULL;
    if (g.rows > 1 && g.ld < g.cols) return MX_ERR_SHAPE;
    if (!aligned(g.data, (uintptr_t)dtype_size(g.dtype))) return MX_ERR_ALIGN;
    // spans and the total stay below 2^62 bytes
    const int64_t pitch = g.rows > 1 ? g.ld : g.cols;
    if (pitch > (((int64_t)1 << 62) / dtype_size(g.dtype)) / g.rows) return MX_ERR_UNSUPPORTED;
    total += g.rows * g.cols;
    if (total > ((int64_t)1 << 60)) return MX_ERR_UNSUPPORTED;
    ++(grad_gapless(g) ? l->gapless : l->gapped);
  }
  // Elements per chunk: enough chunks for every workgroup to walk several, and
  // none so small that looking it up shows: 0.7 M elements 8.5 us with 2048
  // (this rule's), 12.6 us with 32768; 111 M bf16 elements 124 us with 8192
  // (this rule's), 167 us with 2048.
  l->chunk = 2048;
  while (l->chunk < 32768 && total / l->chunk > 16 * mx::kGradGroups) l->chunk *= 2;
  l->chunks = 0;
  for (int32_t i = 0; i < count; ++i)
    l->chunks += (grads[i].rows * grads[i].cols + l->chunk - 1) / l->chunk;
  if (l->chunks > ((int64_t)1 << 31)) return MX_ERR_UNSUPPORTED;
  l->chunks_at = (size_t)count * sizeof(mx::GradTensor);
  l->order_at = l->chunks_at + (size_t)l->chunks * sizeof(mx::GradChunk);
  l->bytes = l->order_at + (size_t)((l->gapless + l->gapped + 1) / 2 * 2) * sizeof(uint32_t);
  return MX_OK;
}

static mx_status check_set(const mx_grad_set *s) {
  if (s == nullptr) return MX_ERR_NULL;
  if (s->count < 0 || s->chunks < 0) return MX_ERR_ARG;
  if (s->count > 0 && s->grads == nullptr) return MX_ERR_NULL;
  if (s->chunks > 0) {
    if (s->host_table == nullptr || s->table == nullptr) return MX_ERR_NULL;
    if (!aligned(s->table, 8)) return MX_ERR_ALIGN;
  }
  return MX_OK;
}

static mx_status check_norm_outputs(const float *norm, const void *workspace, size_t workspace_bytes) {
  if (norm == nullptr || workspace == nullptr) return MX_ERR_NULL;
  if (workspace_bytes < mx_grad_workspace()) return MX_ERR_SHAPE;
  if (!aligned(norm, 4) || !aligned(workspace, 8)) return MX_ERR_ALIGN;
  return MX_OK;
}

static mx::GradTable grad_table(const mx_grad_set *s) {
  mx::GradTable t;
  t.tensors = static_cast<const mx::GradTensor *>(s->table);
  t.chunk_of = reinterpret_cast<const mx::GradChunk *>(static_cast<const uint8_t *>(s->table) +
                                                       (size_t)s->count * sizeof(mx::GradTensor));
  t.chunks = s->chunks;
  t.chunk = s->chunk;
  t.bytes = 0;
  t.once = s->chunks;
  for (int32_t i = 0; i < s->count; ++i) t.bytes += grad_bytes(s->grads[i]);
  return t;
}

// The tensors of a filled set by address, those without gaps and those with.
static void grad_orders(const mx_grad_set *s, GradOrder *without, GradOrder *with) {
  const uint32_t *order = reinterpret_cast<const uint32_t *>(
      static_cast<const uint8_t *>(s->host_table) + (size_t)s->count * sizeof(mx::GradTensor) +
      (size_t)s->chunks * sizeof(mx::GradChunk));
  int64_t n[2] = {0, 0};
  for (int32_t i = 0; i < s->count; ++i)
    if (!grad_empty(s->grads[i])) ++n[grad_gapless(s->grads[i])];
  *without = {s->grads, order, n[1]};
  *with = {s->grads, order + n[1], n[0]};
}

// Whether tensors of two sets of the same shapes share memory other than place
// by place. Those without gaps are merged by address.
static bool grad_sets_clash(const mx_grad_set *a, const mx_grad_set *b) {
  GradOrder x, xg, y, yg;
  grad_orders(a, &x, &xg);
  grad_orders(b, &y, &yg);
  for (int64_t i = 0, j = 0; i < x.n && j < y.n;) {
    const mx_grad &p = a->grads[x.index[i]], &q = b->grads[y.index[j]];
    const uintptr_t pe = address(p) + (uintptr_t)grad_bytes(p);
    const uintptr_t qe = address(q) + (uintptr_t)grad_bytes(q);
    if (pe <= address(q)) {
      ++i;
    } else if (qe <= address(p)) {
      ++j;
    } else {
      if (x.index[i] != y.index[j] || p.data != q.data) return true;
      ++i;
      ++j;
    }
  }
  return any_clash(xg, y) || any_clash(xg, yg) || any_clash(x, yg) || any_clash(yg, x) ||
         any_clash(yg, xg) || any_clash(y, xg);
}

}  // namespace

mx_status mx_grad_set_size(int32_t count, const mx_grad *grads, size_t *table_bytes) {
  if (table_bytes == nullptr) return MX_ERR_NULL;
  GradLayout l;
  const mx_status st = grad_layout(count, grads, &l);
  if (st != MX_OK) return st;
  *table_bytes = l.bytes;
  return MX_OK;
}

mx_status mx_grad_set_fill(int32_t count, const mx_grad *grads, void *host_table,
                           size_t table_bytes, mx_grad_set *set) {
  if (set == nullptr) return MX_ERR_NULL;
  GradLayout l;
  const mx_status st = grad_layout(count, grads, &l);
  if (st != MX_OK) return st;
  if (l.bytes > 0 && host_table == nullptr) return MX_ERR_NULL;
  if (table_bytes < l.bytes) return MX_ERR_SHAPE;
  if (!aligned(host_table, 8)) return MX_ERR_ALIGN;
  uint8_t *base = static_cast<uint8_t *>(host_table);
  uint32_t *order = reinterpret_cast<uint32_t *>(base + l.order_at);
  uint32_t *plain = order, *gaps = order + l.gapless;
  for (int32_t i = 0; i < count; ++i)
    if (!grad_empty(grads[i])) *(grad_gapless(grads[i]) ? plain : gaps)++ = (uint32_t)i;
  auto by_address = [&](uint32_t i, uint32_t j) { return address(grads[i]) < address(grads[j]); };
  std::sort(order, order + l.gapless, by_address);
  std::sort(order + l.gapless, order + l.gapless + l.gapped, by_address);
  for (int64_t i = 1; i < l.gapless; ++i)
    if (address(grads[order[i - 1]]) + (uintptr_t)grad_bytes(grads[order[i - 1]]) >
        address(grads[order[i]]))
      return MX_ERR_ARG;
  const GradOrder without{grads, order, l.gapless}, with{grads, order + l.gapless, l.gapped};
  if (any_clash(with, with) || any_clash(with, without) || any_clash(without, with))
    return MX_ERR_ARG;
  mx::GradTensor *t = reinterpret_cast<mx::GradTensor *>(base);
  mx::GradChunk *c = reinterpret_cast<mx::GradChunk *>(base + l.chunks_at);
  for (int32_t i = 0; i < count; ++i) {
    const mx_grad &g = grads[i];
    t[i].data = g.data;
    t[i].rows = g.rows;
    t[i].cols = g.cols;
    t[i].ld = grad_gapless(g) ? g.cols : g.ld;
    t[i].f32 = g.dtype == MX_OUT_F32 ? 1 : 0;
    const int64_t k = (g.rows * g.cols + l.chunk - 1) / l.chunk;
    for (int64_t j = 0; j < k; ++j) *c++ = mx::GradChunk{(uint32_t)i, (uint32_t)j};
  }
  set->grads = grads;
  set->count = count;
  set->host_table = host_table;
  set->table = nullptr;
  set->table_bytes = l.bytes;
  set->chunks = l.chunks;
  set->chunk = l.chunk;
  return MX_OK;
}

size_t mx_grad_workspace(void) { return mx::kGradGroups * sizeof(double); }

mx_status mx_grad_norm(const mx_grad_set *set, float *norm, void *workspace,
                       size_t workspace_bytes, void *stream) {
  mx_status st = check_set(set);
  if (st != MX_OK) return st;
  st = check_norm_outputs(norm, workspace, workspace_bytes);
  if (st != MX_OK) return st;
  return hip_status(mx::grad_norm_launch(grad_table(set), static_cast<double *>(workspace), norm,
                                         static_cast<hipStream_t>(stream)));
}

mx_status mx_grad_clip(const mx_grad_set *in, const mx_grad_set *out, float max_norm, float *norm,
                       void *workspace, size_t workspace_bytes, void *stream) {
  mx_status st = check_set(in);
  if (st != MX_OK) return st;
  if (out == nullptr) out = in;
  st = check_set(out);
  if (st != MX_OK) return st;
  if (!(max_norm >= 0.0f)) return MX_ERR_ARG;
  if (out != in) {
    if (out->count != in->count || out->chunks != in->chunks || out->chunk != in->chunk)
      return MX_ERR_MISMATCH;
    for (int32_t i = 0; i < in->count; ++i) {
      const mx_grad &p = in->grads[i], &q = out->grads[i];
      if (p.rows != q.rows || p.cols != q.cols || p.dtype != q.dtype) return MX_ERR_MISMATCH;
    }
    if (grad_sets_clash(in, out)) return MX_ERR_ARG;
  }
  st = check_norm_outputs(norm, workspace, workspace_bytes);
  if (st != MX_OK) return st;
  return hip_status(mx::grad_clip_launch(grad_table(in), grad_table(out),
                                         static_cast<double *>(workspace), max_norm, norm,
                                         static_cast<hipStream_t>(stream)));
}

const char *mx_status_string(int32_t status) {
  switch (status) {
    case MX_OK: return "MX_OK";
    case MX_ERR_NULL: return "MX_ERR_NULL: a required pointer is NULL";
    case MX_ERR_SHAPE: return "MX_ERR_SHAPE: bad extents";
    case MX_ERR_ALIGN: return "MX_ERR_ALIGN: misaligned pointer or leading dimension";
    case MX_ERR_ARG: return "MX_ERR_ARG: bad argument value";
    case MX_ERR_MISMATCH: return "MX_ERR_MISMATCH: operands quantized inconsistently";
    case MX_ERR_UNSUPPORTED: return "MX_ERR_UNSUPPORTED: not implemented";
    case MX_ERR_HIP: return "MX_ERR_HIP: HIP runtime error";
    default: return "unknown mx_status";
  }
}

const char *mx_version(void) { return "mxfp4-gfx950 0.1.0"; }

const char *mx_last_hip_error(void) {
  return g_last_hip_error == hipSuccess ? "hipSuccess" : hipGetErrorName(g_last_hip_error);
}

}  // extern "C"
