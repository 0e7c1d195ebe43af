/*
 * lora_mx.h -- microscaled operands of the multi-adapter LoRA linear layer
 * (C ABI, part of liblora_row.so): quantising and reading back, the
 * root-mean-square norm ahead of the projections with a microscaled output,
 * the base product on microscaled operands and the layer on top of them.
 *
 * "Your LoRA Adapters Are Thrashing Your GPUs", section 02: production
 * deployments quantize the base model and keep the LoRA weights in 16 bits.
 * Here the base weight is 4-bit floating point and the activations that meet
 * it are 8- or 4-bit floating point, both with one power-of-two scale for 32
 * consecutive elements of a row, the operand format of CDNA4's scaled matrix
 * instructions (so, unlike with lora_qweight_t, nothing is converted to bf16
 * ahead of the product).  The adapters and their input stay in bf16.
 *
 * Format (OCP Microscaling Formats, version 1.0).  A row of k elements is cut
 * into ceil(k / 32) blocks.  Block b of row i has the scale 2^(s - 127), s =
 * scales[i * lds + b]; element j of the row stands for c_j 2^(s - 127), c_j
 * its code's value:
 *   LORA_MX_FP8: E4M3, byte j of the row (magnitudes 2^-9 .. 448);
 *   LORA_MX_FP4: E2M1, two per byte, element 2i in the low nibble of byte i
 *                (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6).
 * Quantising: s - 127 = max(-127, floor(log2(largest magnitude)) - e), e the
 * exponent of the format's largest code (8, or 2); each element divided by
 * the scale is rounded to the nearest code (ties to even), magnitudes past
 * the largest code take it.  A block that holds an infinity or a NaN gets
 * s = 255 and stands for NaN throughout.  The last block of a row whose
 * length is not a multiple of 32 is filled up with zero codes: a row has
 * ceil(k / 32) * 32 (FP8) or * 16 (FP4) bytes of codes, all of which the
 * library writes and reads.
 * q: device, 16-byte aligned, ldq a multiple of 16 bytes; scales: device,
 * 4-byte aligned, lds a multiple of 4 bytes, >= ceil(k / 32) (the bytes of a
 * row past ceil(k / 32) are not written and may hold anything).
 *
 * Conventions as in lora_row.h: device pointers, row-major, asynchronous on
 * `stream`, errors as lora_status_t, no device allocation, safe to capture
 * into a graph.  M == 0 is a no-op.  Row counts, k and d are at most 2^31 - 1,
 * strides 2^40 bytes, where an operator sets no other limit.
 * lora_profile_* times the product (LORA_K_GEMM) and the layer; quantising,
 * reading back and the norm called by themselves have no class and are not
 * timed.
 */
#ifndef LORA_MX_H
#define LORA_MX_H

#include <stddef.h>
#include <stdint.h>

#include "lora_row.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lora_mxformat {
  LORA_MX_FP8 = 1, /* E4M3, scale per 32 */
  LORA_MX_FP4 = 2  /* E2M1, scale per 32 */
} lora_mxformat_t;

/* A microscaled matrix [rows, k].  The struct is HOST memory, read during the
 * call only. */
typedef struct lora_mx {
  int32_t format;  /* lora_mxformat_t */
  void *q;         /* device, codes [rows, ldq bytes] */
  int64_t ldq;     /* bytes */
  uint8_t *scales; /* device, scale bytes [rows, lds] */
  int64_t lds;     /* bytes */
} lora_mx_t;

/*
 * out = microscaled x.  x [M, k] (ldx >= k; any alignment of its elements'
 * size), dtype F32 or BF16.  out must not overlap x.
 */
lora_status_t lora_mx_quantize(lora_dtype_t dtype, int64_t M, int64_t k, const void *x,
                               int64_t ldx, const lora_mx_t *out, void *stream);

/*
 * y = the values that `in` stands for, in F32 (exact; magnitudes past fp32's
 * largest become infinities) or BF16 (exact where bf16 has the value: always
 * for scales >= 2^-117; else rounded to nearest even).  y [M, k], ldy >= k,
 * must not overlap `in`.
 */
lora_status_t lora_mx_dequantize(lora_dtype_t dtype, int64_t M, int64_t k, const lora_mx_t *in,
                                 void *y, int64_t ldy, void *stream);

/*
 * Root-mean-square norm, with the residual's addition ahead of it:
 *   h = x + residual                               (h = x without a residual)
 *   y[m, j] = h[m, j] / sqrt(mean_j(h[m, j]^2) + eps) * weight[j]
 * residual_out (optional) receives h, y (optional) the normed rows, yq
 * (optional) the normed rows microscaled; y and yq may not both be NULL.
 * Each output is what rounding the 64-bit value once gives, so yq does not
 * depend on whether y is asked for, nor either on how a row was split over
 * threads, but where the last bit of the 64-bit sum decides a tie.  A normed
 * value that fp32 rounds to an infinity is one for yq too: its block gets
 * s = 255.
 * All of x, residual, residual_out, weight and y are of `dtype`.  y and
 * residual_out may each be x or the residual itself (same pointer and
 * leading dimension), not both the same one; other overlaps of an output
 * with an input or another output are LORA_ERR_ARG.
 */
typedef struct lora_norm {
  const void *weight;   /* device [k] */
  float eps;            /* >= 0, finite */
  const void *residual; /* device [M, k], or NULL */
  int64_t ldr;
  void *residual_out; /* device [M, k], or NULL */
  int64_t ldro;
} lora_norm_t;

lora_status_t lora_rmsnorm(lora_dtype_t dtype, int64_t M, int64_t k, const void *x, int64_t ldx,
                           const lora_norm_t *norm, void *y, int64_t ldy, const lora_mx_t *yq,
                           void *stream);

/*
 * y = x W^T on microscaled operands: x [M, k] in FP8 or FP4, W [d, k] in FP4
 * (LORA_ERR_UNSUPPORTED otherwise), y [M, d] bf16 (ldy >= d).  Products and
 * sums run in the scaled matrix instructions with fp32 accumulators; y is
 * rounded once.  Deterministic: the summation order depends on the shape only.
 * Two scales multiply without a range of their own; sums that leave fp32's on
 * the way become infinities or NaNs, as fp32 additions do.  y must not overlap an
 * operand (LORA_ERR_ARG).  ldq and lds of both operands are at most 2^23, so k
 * is at most 2^23 where x is FP8 and 2^24 where it is FP4 (LORA_ERR_SHAPE).
 */
lora_status_t lora_gemm_mx(int64_t M, int64_t k, int64_t d, const lora_mx_t *x,
                           const lora_mx_t *W, void *y, int64_t ldy, void *stream);

/*
 * Testing hook: which of the product's tile shapes a size takes (their order
 * is the library's own; -1: invalid arguments).  Host-only.  out[0], out[1]:
 * the tile's rows of x and of W; out[2]: the elements of k that the longest
 * of the kernel's LDS rings holds (past them all have been refilled).
 */
int32_t lora_test_gemm_mx_shape(int64_t M, int64_t k, int64_t d, int32_t x_format,
                                int32_t out[3]);

/*
 * Bytes of workspace lora_linear_sliced_mx needs for up to max_rows rows (any
 * path, with or without a norm).  Host-only; 0 on invalid arguments.  256-byte
 * aligned, caller-owned, no initialisation needed (nothing here adds to
 * lora_check's n_sync_expired: of a zero-filled workspace it stays 0).
 */
size_t lora_workspace_bytes_sliced_mx(int64_t max_rows, int64_t k, int32_t x_format,
                                      int32_t n_slices, const lora_slice_t *slices);

/*
 * lora_linear_sliced over a microscaled base weight (bf16 x, y, adapters):
 *   xn = x, or with a norm (not NULL) the normed rows of lora_rmsnorm
 *   y[m, :] = quant(xn)[m, :] dequant(W)^T + scale_s (xn[m, :] A_s^T) B_s^T
 * W: FP4, the slices' base weights stacked by rows.  x_format: the format in
 * which xn meets W (lora_mxformat_t); the adapters read xn in bf16.  The base
 * term passes through y in bf16: rows without an adapter are rounded once,
 * adapted ones a second time with the adapter's term added (fp32 sums; xn
 * A_s^T keeps 16 bits or more).  With a norm, residual_out receives x +
 * residual as in lora_rmsnorm; it may be x or the residual itself.  y must not
 * overlap x, the residual or residual_out, nor any of the four the workspace,
 * nor y, residual_out or the workspace W or the norm's weight (LORA_ERR_ARG).
 * Profiling counts the norm or quantising, and the plan beside it, with the
 * product (LORA_K_GEMM).  Everything else as in lora_linear_sliced (k <= 2^23,
 * k, ldx multiples of 8, x 16-byte aligned; lora_check reports on the
 * workspace; up to LORA_PLAN_MAX_ROWS rows those with no adapter equal
 * lora_gemm_mx of the quantised rows bitwise).
 */
lora_status_t lora_linear_sliced_mx(int64_t M, int64_t k, const void *x, int64_t ldx,
                                    const lora_norm_t *norm, int32_t x_format, const lora_mx_t *W,
                                    int32_t n_slices, const lora_slice_t *slices,
                                    const int32_t *adapter_ids, void *y, int64_t ldy,
                                    void *workspace, size_t workspace_bytes, int32_t path,
                                    uint32_t flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_MX_H */
