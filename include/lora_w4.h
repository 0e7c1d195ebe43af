/*
 * lora_w4.h -- a 4-bit base weight with group scales and zero points for the
 * multi-adapter LoRA linear layer (C ABI, part of liblora_row.so): laying the
 * weight out, reading it back, the base product from one row to long prompts,
 * and the layer on top of it.
 *
 * "Your LoRA Adapters Are Thrashing Your GPUs", section 02: production
 * deployments quantize the base model to INT4 and keep the LoRA weights in 16
 * bits.  lora_qweight_t (lora_row.h) is the symmetric form in checkpoint
 * order, for batches; here the codes have a zero point, groups are as small as
 * 32 and need not divide k, and the weight is laid out once, so that one
 * token's product runs at the rate of its bytes.
 *
 * Weight: codes q[n, j] in 0 .. 15; columns j with the same j / group share a
 * scale and a zero point z (a whole number, 0 .. 31):
 *   W[n, j] = scale[n, j / group] (q[n, j] - z[n, j / group])
 * The last group of a row is shorter where `group` does not divide k.
 * group: 32, 64 or a multiple of 128.
 *
 * Conventions as in lora_row.h: device pointers, row-major, asynchronous on
 * `stream`, errors as lora_status_t, no device allocation, safe to capture
 * into a graph.  M == 0 is a no-op.  M, k and d are at most 2^31 - 1 (k here
 * at most 2^24), strides 2^40 bytes.  Products and layers are timed by
 * lora_profile_* (LORA_K_GEMM; the layer's steps under their own classes).
 */
#ifndef LORA_W4_H
#define LORA_W4_H

#include <stddef.h>
#include <stdint.h>

#include "lora_row.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A weight [d, k] as lora_w4_pack lays it out.  The struct is HOST memory,
 * read during the call only. */
typedef struct lora_w4 {
  int32_t group;
  const void *data; /* device, 256-byte aligned, lora_w4_bytes(d, k, group) */
} lora_w4_t;

/* Bytes of a laid-out weight: 4.25 bits a weight (group >= 128; 4.5 with 64, 5
 * with 32), d rounded up to 16 and k to 128.  Host-only; 0 on invalid
 * arguments. */
size_t lora_w4_bytes(int64_t d, int64_t k, int32_t group);

/*
 * Lay out a checkpoint's weight.
 *   q: uint8 [d, ldq], two codes to a byte, column 2i in the low nibble of
 *      byte i; ldq >= ceil(k / 2);
 *   scales: [d, lds] of scale_dtype (F32 or BF16), lds >= ceil(k / group);
 *   zeros: uint8 [d, ldz], ldz >= ceil(k / group), or NULL (8 throughout);
 *      bytes are taken modulo 32.
 * Each scale is kept with 19 significant bits: exact for scales that were
 * bf16 or fp16 before, else rounded to nearest (2^-19 relative).  A NaN or an
 * infinity stays one.  Any alignment of q and zeros.  out must not overlap
 * the others (LORA_ERR_ARG).
 */
lora_status_t lora_w4_pack(int64_t d, int64_t k, int32_t group, const uint8_t *q, int64_t ldq,
                           lora_dtype_t scale_dtype, const void *scales, int64_t lds,
                           const uint8_t *zeros, int64_t ldz, void *out, void *stream);

/*
 * y = W (with the scales as kept), rounded once to F32 or BF16; y [d, k],
 * ldy >= k, any alignment of its elements' size; must not overlap W.
 */
lora_status_t lora_w4_dequantize(lora_dtype_t dtype, int64_t d, int64_t k, const lora_w4_t *W,
                                 void *y, int64_t ldy, void *stream);

/*
 * y = x W^T: x bf16 [M, k] (k, ldx multiples of 8, 16-byte aligned), y bf16
 * [M, d] (ldy >= d).  Up to a number of rows that the weight's sizes alone set
 * (32 at least, up to some hundred for a model's: lora_test_gemm_w4_shape)
 * codes meet x exactly, and each group's sum is scaled and added in fp32; past
 * it the weights are rounded to bf16, once each (by 2^-8 of a weight at most),
 * ahead of the product.  y is rounded once.  Sums that leave fp32's range on the
 * way (|x| past 2^120 or so) and infinities in x may become NaN in their row.
 * Deterministic: the summation order depends on the sizes alone.  y must not
 * overlap x or W (LORA_ERR_ARG).
 */
lora_status_t lora_gemm_w4(int64_t M, int64_t k, int64_t d, const void *x, int64_t ldx,
                           const lora_w4_t *W, void *y, int64_t ldy, void *stream);

/*
 * Testing hook: which of the product's tile shapes a size takes (their order
 * is the library's own; -1: invalid arguments).  Host-only.  out[0], out[1]:
 * the tile's rows of x and of W; out[2]: 1 where it rounds the weights to bf16.
 */
int32_t lora_test_gemm_w4_shape(int64_t M, int64_t k, int64_t d, int32_t group, int32_t out[3]);

/*
 * Bytes of workspace lora_linear_sliced_w4 needs for up to max_rows rows (any
 * path).  Host-only; 0 on invalid arguments.  256-byte aligned, caller-owned,
 * no initialisation needed (but zero-fill it once where lora_check's
 * n_sync_expired is read).
 */
size_t lora_workspace_bytes_sliced_w4(int64_t max_rows, int64_t k, int32_t n_slices,
                                      const lora_slice_t *slices);

/*
 * lora_linear_sliced over such a base weight (bf16 x, y, adapters): W stacks
 * the slices' base weights by rows.  Everything else as in lora_linear_sliced.
 * Rows without an adapter are lora_gemm_w4's, bit for bit (up to 8192 rows,
 * which one plan holds).  Up to 32 rows (but by LORA_PATH_GATHER) need no plan,
 * round y once and keep 16 bits of each rank's product between A and B; they
 * leave a plan for others unless LORA_FLAG_REUSE_PLAN is given.  More rows round
 * the base product to y and then its sum with the adapters' part, as the other
 * layers do.  y must not overlap x, W or the workspace (LORA_ERR_ARG).
 */
lora_status_t lora_linear_sliced_w4(int64_t M, int64_t k, const void *x, int64_t ldx,
                                    const lora_w4_t *W, int32_t n_slices,
                                    const lora_slice_t *slices, const int32_t *adapter_ids, void *y,
                                    int64_t ldy, void *workspace, size_t workspace_bytes,
                                    int32_t path, uint32_t flags, void *stream);

/*
 * Testing hook: which product lora_linear_sliced_w4 (but by LORA_PATH_GATHER)
 * launches for 1 to 8192 rows without a given plan: of those that add the
 * adapters' part, numbered first, or of lora_gemm_w4's (-1: invalid arguments).
 * Host-only.  out[0], out[1]: the tile's rows of x and of W; out[2]: 1 where the
 * plan is made in its launch.
 */
int32_t lora_test_linear_w4_shape(int64_t M, int64_t k, int64_t d, int32_t group, int32_t out[3]);

#ifdef __cplusplus
}
#endif

#endif /* LORA_W4_H */
