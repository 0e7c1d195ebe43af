// w4_api.cpp -- host side of include/lora_w4.h: argument checks and launches
// (the layer runs in lora_api.cpp's linear_sliced_impl).
#include <hip/hip_runtime.h>

#include "lora_w4.h"
#include "kernels.hpp"
#include "spans.hpp"

namespace lora {

namespace {

constexpr int64_t kMaxK = int64_t(1) << 24;
constexpr int64_t kMaxBytes = int64_t(1) << 40;

int64_t records(int64_t k) { return (k + 127) / 128; }
int32_t groups_in_record(int32_t group) { return group >= 128 ? 1 : 128 / group; }

lora_status_t check_w4(int64_t d, int64_t k, const lora_w4_t *W) {
  if (W == nullptr) return LORA_ERR_ARG;
  if (lora_w4_bytes(d, k, W->group) == 0) return LORA_ERR_SHAPE;
  if (W->data == nullptr) return LORA_ERR_ARG;
  if ((uintptr_t)W->data % 256 != 0) return LORA_ERR_SHAPE;
  return LORA_OK;
}

Span w4_span(int64_t d, int64_t k, int32_t group, const void *data) {
  const int64_t n = (int64_t)lora_w4_bytes(d, k, group);
  return Span{(const uint8_t *)data, n, n};
}

W4Args w4_args(int64_t d, int64_t k, int32_t group) {
  W4Args a{};
  a.d = d;
  a.k = k;
  a.group = group;
  a.nb = (int32_t)records(k);
  a.sg = groups_in_record(group);
  return a;
}

}  // namespace

lora_status_t check_gemm_w4(int64_t M, int64_t k, int64_t d, const void *x, int64_t ldx,
                            const lora_w4_t *W, const void *y, int64_t ldy, const void *workspace,
                            size_t workspace_bytes) {
  if (M < 0 || M > INT32_MAX || d < 1 || k < 1) return LORA_ERR_SHAPE;
  lora_status_t s = check_w4(d, k, W);
  if (s != LORA_OK || M == 0) return s;
  if ((s = check_dense(LORA_DTYPE_BF16, k, x, ldx)) != LORA_OK) return s;
  if (k % 8 || ldx % 8 || (uintptr_t)x % 16) return LORA_ERR_SHAPE;
  if ((s = check_dense(LORA_DTYPE_BF16, d, y, ldy)) != LORA_OK) return s;
  const Span out = dense_span(LORA_DTYPE_BF16, d, y, ldy), in = dense_span(LORA_DTYPE_BF16, k, x, ldx);
  const Span w = w4_span(d, k, W->group, W->data);
  // an empty range shares no byte with anything
  const Span ws{workspace_bytes > 0 ? (const uint8_t *)workspace : nullptr, (int64_t)workspace_bytes,
                (int64_t)workspace_bytes};
  if (overlap(out, in, M) || meet(out, M, w, 1) || meet(out, M, ws, 1) || meet(in, M, ws, 1) || meet(w, 1, ws, 1))
    return LORA_ERR_ARG;
  return LORA_OK;
}

W4GemmArgs make_w4_args(int64_t M, int64_t k, int64_t d, const void *x, int64_t ldx,
                        const lora_w4_t *W, void *y, int64_t ldy) {
  W4GemmArgs a{};
  a.M = (int32_t)M;
  a.N = (int32_t)d;
  a.K = (int32_t)k;
  a.nb = (int32_t)records(k);
  a.sg = groups_in_record(W->group);
  a.x = (const uint16_t *)x;
  a.ldx = ldx;
  a.w = (const uint8_t *)W->data;
  a.y = (uint16_t *)y;
  a.ldy = ldy;
  return a;
}

}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_w4_bytes(int64_t d, int64_t k, int32_t group) {
  if (d < 1 || d > INT32_MAX || k < 1 || k > kMaxK) return 0;
  if (group != 32 && group != 64 && (group < 128 || group % 128 != 0)) return 0;
  const int64_t n = (d + 15) / 16 * records(k) * w4_record(groups_in_record(group));
  return n <= kMaxBytes ? (size_t)n : 0;
}

lora_status_t lora_w4_pack(int64_t d, int64_t k, int32_t group, const uint8_t *q, int64_t ldq,
                           lora_dtype_t scale_dtype, const void *scales, int64_t lds,
                           const uint8_t *zeros, int64_t ldz, void *out, void *stream) {
  if (scale_dtype != LORA_DTYPE_F32 && scale_dtype != LORA_DTYPE_BF16) return LORA_ERR_DTYPE;
  const size_t bytes = lora_w4_bytes(d, k, group);
  if (bytes == 0) return LORA_ERR_SHAPE;
  if (q == nullptr || scales == nullptr || out == nullptr) return LORA_ERR_ARG;
  const int64_t ng = (k + group - 1) / group;
  if (ldq < (k + 1) / 2 || ldq > kMaxLd || (uintptr_t)out % 256 != 0) return LORA_ERR_SHAPE;
  if (zeros != nullptr && (ldz < ng || ldz > kMaxLd)) return LORA_ERR_SHAPE;
  lora_status_t s = check_dense(scale_dtype, ng, scales, lds);
  if (s != LORA_OK) return s;
  const Span o = w4_span(d, k, group, out);
  if (meet(o, 1, Span{q, ldq, (k + 1) / 2}, d) || meet(o, 1, dense_span(scale_dtype, ng, scales, lds), d) ||
      meet(o, 1, Span{zeros, ldz, ng}, d))
    return LORA_ERR_ARG;
  W4Args a = w4_args(d, k, group);
  a.q = q;
  a.ldq = ldq;
  a.scale_dtype = scale_dtype;
  a.scales = scales;
  a.lds = lds;
  a.zeros = zeros;
  a.ldz = ldz;
  a.w = (uint8_t *)out;
  return launch_w4_pack(a, (hipStream_t)stream) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status_t lora_w4_dequantize(lora_dtype_t dtype, int64_t d, int64_t k, const lora_w4_t *W,
                                 void *y, int64_t ldy, void *stream) {
  if (dtype != LORA_DTYPE_F32 && dtype != LORA_DTYPE_BF16) return LORA_ERR_DTYPE;
  if (d < 1 || k < 1) return LORA_ERR_SHAPE;
  lora_status_t s = check_w4(d, k, W);
  if (s != LORA_OK) return s;
  if ((s = check_dense(dtype, k, y, ldy)) != LORA_OK) return s;
  if (meet(dense_span(dtype, k, y, ldy), d, w4_span(d, k, W->group, W->data), 1)) return LORA_ERR_ARG;
  W4Args a = w4_args(d, k, W->group);
  a.w = (uint8_t *)W->data;
  a.dtype = dtype;
  a.y = y;
  a.ldy = ldy;
  return launch_w4_dequantize(a, (hipStream_t)stream) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status_t lora_gemm_w4(int64_t M, int64_t k, int64_t d, const void *x, int64_t ldx,
                           const lora_w4_t *W, void *y, int64_t ldy, void *stream) {
  const lora_status_t s = check_gemm_w4(M, k, d, x, ldx, W, y, ldy, nullptr, 0);
  if (s != LORA_OK || M == 0) return s;
  const hipError_t e = timed(LORA_K_GEMM, (hipStream_t)stream,
                             [&] { return launch_gemm_w4(make_w4_args(M, k, d, x, ldx, W, y, ldy), (hipStream_t)stream); });
  return e == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

int32_t lora_test_gemm_w4_shape(int64_t M, int64_t k, int64_t d, int32_t group, int32_t out[3]) {
  if (out == nullptr || M < 1 || lora_w4_bytes(d, k, group) == 0) return -1;
  return gemm_w4_shape(M, k, d, groups_in_record(group), out);
}

int32_t lora_test_linear_w4_shape(int64_t M, int64_t k, int64_t d, int32_t group, int32_t out[3]) {
  if (out == nullptr || M < 1 || M > kPlanMaxRows || k % 8 || lora_w4_bytes(d, k, group) == 0) return -1;
  const lora_w4_t W{group, nullptr};
  return linear_w4_shape(make_w4_args(M, k, d, nullptr, k, &W, nullptr, d), out);
}

size_t lora_workspace_bytes_sliced_w4(int64_t max_rows, int64_t k, int32_t n_slices,
                                      const lora_slice_t *slices) {
  if (k < 1 || k > kMaxK) return 0;
  // the plan's regions alone, which depend on no type: in fp32 the dense base
  // product, which this layer does not run, takes none of its own
  return lora_workspace_bytes_sliced(max_rows, k, LORA_DTYPE_F32, n_slices, slices);
}

lora_status_t lora_linear_sliced_w4(int64_t M, int64_t k, const void *x, int64_t ldx,
                                    const lora_w4_t *W, int32_t n_slices,
                                    const lora_slice_t *slices, const int32_t *adapter_ids, void *y,
                                    int64_t ldy, void *workspace, size_t workspace_bytes,
                                    int32_t path, uint32_t flags, void *stream) {
  const W4Base w4{W};
  return linear_sliced_impl(LORA_DTYPE_BF16, M, k, x, ldx, nullptr, 0, nullptr, n_slices, slices,
                            adapter_ids, y, ldy, workspace, workspace_bytes, path, flags, stream,
                            false, nullptr, &w4);
}

}  // extern "C"
