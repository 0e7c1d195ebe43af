/*
 * lora_heads.h -- the step behind the query and key projections (C ABI, part
 * of liblora_row.so): the root-mean-square norm of each head and the rotation
 * by its position, in one pass.
 *
 * "Your LoRA Adapters Are Thrashing Your GPUs", section 02 (the query and
 * value projections are the usual adapted pair): the projections' output goes
 * on as heads.  For each row m and head h of q, and of k:
 *   u[j] = x[m, h, j] / sqrt(mean_j(x[m, h, j]^2) + eps) * weight[j]
 *          (u = x where the weight is NULL)
 *   (u[a], u[b]) -> (u[a] c - u[b] s, u[b] c + u[a] s),  i < rot_dim / 2,
 *          c = scale cos(positions[m] inv_freq[i]), s likewise with sin
 * with a, b = i, i + rot_dim / 2, or interleaved 2i, 2i + 1; columns from
 * rot_dim on keep u.
 *
 * Conventions as in lora_row.h (device pointers, strides in elements,
 * asynchronous on `stream`, lora_status_t, no device allocation, safe to
 * capture).  M == 0 is a no-op.  Not timed by lora_profile_*.
 */
#ifndef LORA_HEADS_H
#define LORA_HEADS_H

#include <stdint.h>

#include "lora_row.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Heads of one kind: element j of head h of row m is x[m * ld_row + h *
 * ld_head + j], and likewise in out.  The struct is HOST memory. */
typedef struct lora_heads {
  int32_t n_heads;
  const void *x;
  int64_t ld_row, ld_head;
  const void *weight; /* device [head_dim], or NULL: no norm */
  void *out;          /* x itself (same strides), or memory apart from every input */
  int64_t ldo_row, ldo_head;
} lora_heads_t;

/* The rotation.  The struct is HOST memory. */
typedef struct lora_rope {
  const int64_t *positions; /* device [M] */
  const float *inv_freq;    /* device [rot_dim / 2] */
  int32_t rot_dim;          /* even, 2 .. head_dim */
  int32_t interleaved;      /* 0 or 1 */
  float scale;              /* of cos and sin; finite */
} lora_rope_t;

/*
 * q: not NULL; k, rope: may be NULL (no keys; norms alone).  All tensors but
 * positions and inv_freq are of `dtype` (F32 or BF16), aligned to their
 * elements; head_dim 1 .. 1024, n_heads 1 .. 65535, strides below 2^40;
 * rows and heads of a tensor must not overlap one another: ld_head, ld_row >=
 * head_dim, and ld_row >= (n_heads - 1) ld_head + head_dim (all heads of a row,
 * then the next row) or ld_head >= (M - 1) ld_row + head_dim (all rows of a
 * head, then the next head); ld_head counts only where n_heads > 1, ld_row
 * where M > 1.  Sums of squares and angles
 * are computed in 64 bits, the values in fp32 (two roundings of the norm, three
 * of the rotation); each output is rounded once from there.  A row whose
 * position is negative (padding) is left as it is in both outputs.  The
 * angle is exact to 2^-50 of itself: to fp32's last bit for positions below
 * 2^26.  A q or k `out` over an input other than its own x, or over the other
 * output, is LORA_ERR_ARG.
 */
lora_status_t lora_qk_norm_rope(lora_dtype_t dtype, int64_t M, int32_t head_dim, float eps,
                                const lora_heads_t *q, const lora_heads_t *k,
                                const lora_rope_t *rope, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_HEADS_H */
