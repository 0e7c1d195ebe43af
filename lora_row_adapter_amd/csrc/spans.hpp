// spans.hpp -- host checks of dense tensors and of what may overlap, shared by
// the entry points (internal to liblora_row).
#pragma once

#include <stdint.h>

#include "lora_row.h"

namespace lora {

constexpr int64_t kMaxLd = int64_t(1) << 40;  // leading dimensions, in bytes
inline int64_t elem_bytes(lora_dtype_t t) { return t == LORA_DTYPE_BF16 ? 2 : 4; }

// Runs of `width` bytes, `ld` bytes apart.
struct Span {
  const uint8_t *p;
  int64_t ld, width;
};
// Past its last byte, with as many rows as that (no product of a caller's
// numbers wraps).
inline unsigned __int128 end_of(const Span &s, int64_t rows) {
  return (unsigned __int128)(uintptr_t)s.p + (unsigned __int128)(rows - 1) * (unsigned __int128)s.ld + s.width;
}
inline bool meet(const Span &a, int64_t rows_a, const Span &b, int64_t rows_b) {
  return a.p != nullptr && b.p != nullptr && end_of(a, rows_a) > (uintptr_t)b.p && end_of(b, rows_b) > (uintptr_t)a.p;
}
// Whether two such regions share a byte.  With equal strides the runs are
// compared inside one stride (columns of one wide buffer do not overlap);
// with different ones the whole ranges are.
inline bool overlap(const Span &a, const Span &b, int64_t rows) {
  if (!meet(a, rows, b, rows)) return false;
  if (a.ld == b.ld && rows > 1) {
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const int64_t o = (int64_t)((b0 >= a0 ? b0 - a0 : a0 - b0) % (uintptr_t)a.ld);
    const int64_t first = b0 >= a0 ? a.width : b.width, second = b0 >= a0 ? b.width : a.width;
    return o < first || o + second > a.ld;
  }
  return true;
}
inline bool same(const Span &a, const Span &b) { return a.p == b.p && a.ld == b.ld; }

// A dense matrix of `dtype`: set, rows long enough, elements aligned.
inline lora_status_t check_dense(lora_dtype_t dtype, int64_t k, const void *p, int64_t ld) {
  if (p == nullptr) return LORA_ERR_ARG;
  const int64_t eb = elem_bytes(dtype);
  if (ld < k || ld > kMaxLd / eb || (uintptr_t)p % eb != 0) return LORA_ERR_SHAPE;
  return LORA_OK;
}

inline Span dense_span(lora_dtype_t dtype, int64_t k, const void *p, int64_t ld) {
  const int64_t eb = elem_bytes(dtype);
  return Span{(const uint8_t *)p, ld * eb, k * eb};
}

}  // namespace lora
