// mx_api.cpp -- host side of include/lora_mx.h: argument checks and launches
// (the microscaled layer itself runs in lora_api.cpp's linear_sliced_impl).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "lora_mx.h"
#include "kernels.hpp"
#include "spans.hpp"

namespace lora {

namespace {

int64_t blocks_of(int64_t k) { return (k + 31) / 32; }
int64_t code_bytes(int32_t fmt, int64_t k) { return blocks_of(k) * (fmt == LORA_MX_FP8 ? 32 : 16); }

lora_status_t check_sizes(lora_dtype_t dtype, int64_t M, int64_t k) {
  if (dtype != LORA_DTYPE_F32 && dtype != LORA_DTYPE_BF16) return LORA_ERR_DTYPE;
  if (M < 0 || k < 1 || M > INT32_MAX || k > INT32_MAX) return LORA_ERR_SHAPE;
  return LORA_OK;
}

Span code_span(const lora_mx_t *m, int64_t k) {
  return Span{(const uint8_t *)m->q, m->ldq, code_bytes(m->format, k)};
}
Span scale_span(const lora_mx_t *m, int64_t k) { return Span{m->scales, m->lds, blocks_of(k)}; }

// Whether an output of the norm keeps apart from the weight and from x and
// the residual -- or, with in_place, is exactly one of those two.
bool norm_output_apart(lora_dtype_t dtype, int64_t M, int64_t k, const void *x, int64_t ldx,
                       const lora_norm_t *n, const Span &out, bool in_place) {
  if (out.p == nullptr) return true;
  for (const Span &v : {dense_span(dtype, k, x, ldx), dense_span(dtype, k, n->residual, n->ldr)})
    if (overlap(out, v, M) && !(in_place && same(out, v))) return false;
  // the weight is one row: no row of the output may meet it
  return !meet(out, M, dense_span(dtype, k, n->weight, k), 1);
}

lora_status_t quant_args(lora_dtype_t dtype, int64_t M, int64_t k, const void *x, int64_t ldx,
                         const lora_mx_t *q, MxQuantArgs *a) {
  lora_status_t s = check_sizes(dtype, M, k);
  if (s != LORA_OK) return s;
  s = check_mx(q, M, k);
  if (s != LORA_OK || M == 0) return s;
  s = check_dense(dtype, k, x, ldx);
  if (s != LORA_OK) return s;
  const Span d = dense_span(dtype, k, x, ldx), c = code_span(q, k), e = scale_span(q, k);
  if (overlap(d, c, M) || overlap(d, e, M) || overlap(c, e, M)) return LORA_ERR_ARG;
  a->dtype = dtype;
  a->fmt = q->format;
  a->M = M;
  a->k = k;
  a->x = x;
  a->ldx = ldx;
  a->q = (uint8_t *)q->q;
  a->ldq = q->ldq;
  a->sc = q->scales;
  a->lds = q->lds;
  return LORA_OK;
}

}  // namespace

lora_status_t check_mx(const lora_mx_t *m, int64_t rows, int64_t k) {
  if (m == nullptr) return LORA_ERR_ARG;
  if (m->format != LORA_MX_FP8 && m->format != LORA_MX_FP4) return LORA_ERR_DTYPE;
  if (rows == 0) return LORA_OK;
  if (m->q == nullptr || m->scales == nullptr) return LORA_ERR_ARG;
  if ((uintptr_t)m->q % 16 != 0 || m->ldq % 16 != 0) return LORA_ERR_SHAPE;
  if ((uintptr_t)m->scales % 4 != 0 || m->lds % 4 != 0) return LORA_ERR_SHAPE;
  if (m->ldq < code_bytes(m->format, k) || m->lds < blocks_of(k)) return LORA_ERR_SHAPE;
  if (m->ldq > kMaxLd || m->lds > kMaxLd) return LORA_ERR_SHAPE;
  return LORA_OK;
}

lora_status_t check_norm_in(lora_dtype_t dtype, int64_t M, int64_t k, const void *x, int64_t ldx,
                            const lora_norm_t *n) {
  lora_status_t s = check_sizes(dtype, M, k);
  if (s != LORA_OK) return s;
  if (n == nullptr || !(n->eps >= 0.f) || std::isinf(n->eps)) return LORA_ERR_ARG;
  if (M == 0) return LORA_OK;
  if ((s = check_dense(dtype, k, x, ldx)) != LORA_OK) return s;
  if ((s = check_dense(dtype, k, n->weight, k)) != LORA_OK) return s;
  if (n->residual != nullptr && (s = check_dense(dtype, k, n->residual, n->ldr)) != LORA_OK) return s;
  if (n->residual_out == nullptr) return LORA_OK;
  if ((s = check_dense(dtype, k, n->residual_out, n->ldro)) != LORA_OK) return s;
  return norm_output_apart(dtype, M, k, x, ldx, n, dense_span(dtype, k, n->residual_out, n->ldro), true)
             ? LORA_OK
             : LORA_ERR_ARG;
}

lora_status_t check_norm(lora_dtype_t dtype, int64_t M, int64_t k, const void *x, int64_t ldx,
                         const lora_norm_t *n, const void *y, int64_t ldy, const lora_mx_t *yq) {
  lora_status_t s = check_norm_in(dtype, M, k, x, ldx, n);
  if (s != LORA_OK) return s;
  if (y == nullptr && yq == nullptr) return LORA_ERR_ARG;
  if (yq != nullptr && (s = check_mx(yq, M, k)) != LORA_OK) return s;
  if (M == 0) return LORA_OK;
  if (y != nullptr && (s = check_dense(dtype, k, y, ldy)) != LORA_OK) return s;
  const Span none{nullptr, 0, 0};
  const Span out[4] = {dense_span(dtype, k, n->residual_out, n->ldro), dense_span(dtype, k, y, ldy),
                       yq ? code_span(yq, k) : none, yq ? scale_span(yq, k) : none};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (overlap(out[i], out[j], M)) return LORA_ERR_ARG;
  for (int i = 1; i < 4; ++i)
    if (!norm_output_apart(dtype, M, k, x, ldx, n, out[i], i == 1)) return LORA_ERR_ARG;
  return LORA_OK;
}

lora_status_t check_gemm_mx(int64_t M, int64_t k, int64_t d, const lora_mx_t *W) {
  if (M < 0 || k < 1 || d < 1) return LORA_ERR_SHAPE;
  if (M > INT32_MAX || k > INT32_MAX - 512 || d > INT32_MAX) return LORA_ERR_SHAPE;
  const lora_status_t s = check_mx(W, d, k);
  if (s != LORA_OK) return s;
  if (W->format != LORA_MX_FP4) return LORA_ERR_UNSUPPORTED;
  // offsets inside one tile's rows are 32 bits wide
  if (W->ldq > (int64_t(1) << 23) || W->lds > (int64_t(1) << 23)) return LORA_ERR_SHAPE;
  return LORA_OK;
}

lora_status_t check_layer_apart(int64_t M, int64_t k, int64_t d, const void *x, int64_t ldx,
                                const lora_norm_t *n, const lora_mx_t *W, const void *y, int64_t ldy,
                                const void *workspace, size_t workspace_bytes) {
  const lora_status_t s = check_dense(LORA_DTYPE_BF16, d, y, ldy);
  if (s != LORA_OK) return s;
  if (ldx > kMaxLd / 2) return LORA_ERR_SHAPE;
  const Span out = dense_span(LORA_DTYPE_BF16, d, y, ldy);
  const Span ws{(const uint8_t *)workspace, (int64_t)workspace_bytes, (int64_t)workspace_bytes};
  Span others[3] = {dense_span(LORA_DTYPE_BF16, k, x, ldx), {}, {}};
  if (n != nullptr) {
    others[1] = dense_span(LORA_DTYPE_BF16, k, n->residual, n->ldr);
    others[2] = dense_span(LORA_DTYPE_BF16, k, n->residual_out, n->ldro);
  }
  if (meet(out, M, ws, 1)) return LORA_ERR_ARG;
  for (const Span &o : others)
    if (overlap(out, o, M) || meet(o, M, ws, 1)) return LORA_ERR_ARG;
  // (the norm's sum keeps apart from its weight: check_norm_in)
  const Span weight = n != nullptr ? dense_span(LORA_DTYPE_BF16, k, n->weight, k) : Span{};
  if (meet(weight, 1, out, M) || meet(weight, 1, ws, 1)) return LORA_ERR_ARG;
  for (const Span &w : {code_span(W, k), scale_span(W, k)})
    if (meet(w, d, out, M) || meet(w, d, ws, 1) || meet(w, d, others[2], M)) return LORA_ERR_ARG;
  return LORA_OK;
}

MxLayout mx_layout(int64_t rows, int64_t k, int32_t x_format) {
  MxLayout L;
  L.ldq = code_bytes(x_format, k);
  L.lds = (blocks_of(k) + 3) & ~int64_t(3);
  L.ldn = (k + 7) & ~int64_t(7);
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  L.q = 0;
  L.sc = up((size_t)(rows * L.ldq));
  L.xn = L.sc + up((size_t)(rows * L.lds));
  L.total = L.xn + up((size_t)(rows * L.ldn * 2));
  return L;
}

}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_mx_quantize(lora_dtype_t dtype, int64_t M, int64_t k, const void *x,
                               int64_t ldx, const lora_mx_t *out, void *stream) {
  MxQuantArgs a{};
  const lora_status_t s = quant_args(dtype, M, k, x, ldx, out, &a);
  if (s != LORA_OK || M == 0) return s;
  return launch_mx_quantize(a, (hipStream_t)stream) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status_t lora_mx_dequantize(lora_dtype_t dtype, int64_t M, int64_t k, const lora_mx_t *in,
                                 void *y, int64_t ldy, void *stream) {
  MxQuantArgs a{};
  const lora_status_t s = quant_args(dtype, M, k, y, ldy, in, &a);
  if (s != LORA_OK || M == 0) return s;
  return launch_mx_dequantize(a, (hipStream_t)stream) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status_t lora_rmsnorm(lora_dtype_t dtype, int64_t M, int64_t k, const void *x, int64_t ldx,
                           const lora_norm_t *norm, void *y, int64_t ldy, const lora_mx_t *yq,
                           void *stream) {
  const lora_status_t s = check_norm(dtype, M, k, x, ldx, norm, y, ldy, yq);
  if (s != LORA_OK || M == 0) return s;
  RmsNormArgs a{};
  a.dtype = dtype;
  a.M = M;
  a.k = k;
  a.x = x;
  a.ldx = ldx;
  a.res = norm->residual;
  a.ldr = norm->ldr;
  a.w = norm->weight;
  a.h = norm->residual_out;
  a.ldh = norm->ldro;
  a.y = y;
  a.ldy = ldy;
  a.eps = norm->eps;
  if (yq != nullptr) {
    a.fmt = yq->format;
    a.q = (uint8_t *)yq->q;
    a.ldq = yq->ldq;
    a.sc = yq->scales;
    a.lds = yq->lds;
  }
  return launch_rmsnorm(a, (hipStream_t)stream) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status_t lora_gemm_mx(int64_t M, int64_t k, int64_t d, const lora_mx_t *x,
                           const lora_mx_t *W, void *y, int64_t ldy, void *stream) {
  lora_status_t s = check_gemm_mx(M, k, d, W);
  if (s != LORA_OK) return s;
  if ((s = check_mx(x, M, k)) != LORA_OK || M == 0) return s;
  if (x->ldq > (int64_t(1) << 23) || x->lds > (int64_t(1) << 23)) return LORA_ERR_SHAPE;
  if ((s = check_dense(LORA_DTYPE_BF16, d, y, ldy)) != LORA_OK) return s;
  const Span out = dense_span(LORA_DTYPE_BF16, d, y, ldy);
  if (meet(out, M, code_span(x, k), M) || meet(out, M, scale_span(x, k), M) ||
      meet(out, M, code_span(W, k), d) || meet(out, M, scale_span(W, k), d))
    return LORA_ERR_ARG;
  MxGemmArgs a{};
  a.xfmt = x->format;
  a.M = (int32_t)M;
  a.N = (int32_t)d;
  a.nb = (int32_t)blocks_of(k);
  a.x = (const uint8_t *)x->q;
  a.ldx = x->ldq;
  a.xs = x->scales;
  a.ldxs = x->lds;
  a.w = (const uint8_t *)W->q;
  a.ldw = W->ldq;
  a.wsc = W->scales;
  a.ldws = W->lds;
  a.y = (uint16_t *)y;
  a.ldy = ldy;
  const hipError_t e = timed(LORA_K_GEMM, (hipStream_t)stream, [&] { return launch_gemm_mx(a, (hipStream_t)stream); });
  return e == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

int32_t lora_test_gemm_mx_shape(int64_t M, int64_t k, int64_t d, int32_t x_format, int32_t out[3]) {
  if (x_format != LORA_MX_FP8 && x_format != LORA_MX_FP4) return -1;
  if (out == nullptr || M < 1 || d < 1 || k < 1 || k > INT32_MAX - 512) return -1;
  return gemm_mx_shape(M, k, d, x_format, out);
}

size_t lora_workspace_bytes_sliced_mx(int64_t max_rows, int64_t k, int32_t x_format,
                                      int32_t n_slices, const lora_slice_t *slices) {
  if (x_format != LORA_MX_FP8 && x_format != LORA_MX_FP4) return 0;
  if (max_rows < 0 || k < 1 || k > INT32_MAX) return 0;
  // the plan's regions alone, which depend on no type: in fp32 the dense base
  // product, which this layer does not run, takes none of its own
  const size_t plan = lora_workspace_bytes_sliced(max_rows, k, LORA_DTYPE_F32, n_slices, slices);
  if (plan == 0) return 0;
  const int64_t rows = std::min<int64_t>(std::max<int64_t>(max_rows, 1), kPlanMaxRows);
  return plan + mx_layout(rows, k, x_format).total;
}

lora_status_t lora_linear_sliced_mx(int64_t M, int64_t k, const void *x, int64_t ldx,
                                    const lora_norm_t *norm, int32_t x_format, const lora_mx_t *W,
                                    int32_t n_slices, const lora_slice_t *slices,
                                    const int32_t *adapter_ids, void *y, int64_t ldy,
                                    void *workspace, size_t workspace_bytes, int32_t path,
                                    uint32_t flags, void *stream) {
  const MxBase mx{W, x_format, norm};
  return linear_sliced_impl(LORA_DTYPE_BF16, M, k, x, ldx, nullptr, 0, nullptr, n_slices, slices,
                            adapter_ids, y, ldy, workspace, workspace_bytes, path, flags, stream,
                            false, &mx);
}

}  // extern "C"
