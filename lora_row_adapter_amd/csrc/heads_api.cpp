// heads_api.cpp -- host side of include/lora_heads.h: argument checks.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "lora_heads.h"
#include "kernels.hpp"
#include "spans.hpp"

namespace lora {

namespace {

typedef __int128 wide;

// Elements [p + m ld_row + h ld_head, + D) for m < M, h < H, in bytes.
struct Region {
  uintptr_t p;
  int64_t row, head, D;
  int64_t M, H;
};
Region region(const void *p, int64_t row, int64_t head, int64_t D, int64_t M, int64_t H, int64_t eb) {
  return Region{(uintptr_t)p, M > 1 ? row * eb : 0, H > 1 ? head * eb : 0, D * eb, M, H};
}
wide end_of(const Region &r) {
  return (wide)r.p + (wide)(r.M - 1) * r.row + (wide)(r.H - 1) * r.head + r.D;
}
// Whether two regions share a byte: exactly where their strides agree (heads
// of q and of k in one wide buffer), else by their whole ranges.
bool overlap(const Region &a, const Region &b) {
  if (a.p == 0 || b.p == 0) return false;
  if (end_of(a) <= (wide)b.p || end_of(b) <= (wide)a.p) return false;
  const int64_t row = std::max(a.row, b.row), head = std::max(a.head, b.head);
  if ((a.row != 0 && a.row != row) || (b.row != 0 && b.row != row)) return true;
  if ((a.head != 0 && a.head != head) || (b.head != 0 && b.head != head)) return true;
  // head hb of b lies dh heads after head ha of a; the rows between them, if
  // any, that bring the two within a head of each other
  for (int64_t dh = -(a.H - 1); dh <= b.H - 1; ++dh) {
    const wide o = (wide)b.p - (wide)a.p + (wide)dh * head;
    wide dm = 0;
    if (row > 0) {
      dm = -o / row;
      dm = std::max<wide>(-(wide)(a.M - 1), std::min<wide>(b.M - 1, dm));
    }
    for (wide i = std::max<wide>(dm - 1, -(wide)(a.M - 1)); i <= std::min<wide>(dm + 1, b.M - 1); ++i) {
      const wide at = o + i * row;
      if (at < a.D && -at < b.D) return true;
    }
  }
  return false;
}

lora_status_t check_strides(int64_t M, int64_t H, int64_t D, int64_t row, int64_t head) {
  if ((M > 1 && (row < D || row >= kMaxLd)) || (H > 1 && (head < D || head >= kMaxLd))) return LORA_ERR_SHAPE;
  // rows of all heads one after another, or heads of all rows
  if (M > 1 && H > 1 && row < (wide)(H - 1) * head + D && head < (wide)(M - 1) * row + D) return LORA_ERR_SHAPE;
  return LORA_OK;
}

lora_status_t check_heads(int64_t M, int64_t D, int64_t eb, const lora_heads_t *h) {
  if (h->n_heads < 1 || h->n_heads > 65535) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  if (h->x == nullptr || h->out == nullptr) return LORA_ERR_ARG;
  if ((uintptr_t)h->x % eb || (uintptr_t)h->out % eb || (uintptr_t)h->weight % eb) return LORA_ERR_SHAPE;
  const lora_status_t s = check_strides(M, h->n_heads, D, h->ld_row, h->ld_head);
  return s != LORA_OK ? s : check_strides(M, h->n_heads, D, h->ldo_row, h->ldo_head);
}

bool in_place(int64_t M, const lora_heads_t *h) {
  return h->x == h->out && (M == 1 || h->ld_row == h->ldo_row) && (h->n_heads == 1 || h->ld_head == h->ldo_head);
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_qk_norm_rope(lora_dtype_t dtype, int64_t M, int32_t head_dim, float eps,
                                const lora_heads_t *q, const lora_heads_t *k,
                                const lora_rope_t *rope, void *stream) {
  if (dtype != LORA_DTYPE_F32 && dtype != LORA_DTYPE_BF16) return LORA_ERR_DTYPE;
  if (M < 0 || M > INT32_MAX || head_dim < 1 || head_dim > 1024) return LORA_ERR_SHAPE;
  if (q == nullptr || !(eps >= 0.f) || std::isinf(eps)) return LORA_ERR_ARG;
  const int64_t eb = elem_bytes(dtype), D = head_dim;
  const lora_heads_t *sets[2] = {q, k};
  for (const lora_heads_t *h : sets) {
    if (h == nullptr) continue;
    const lora_status_t s = check_heads(M, D, eb, h);
    if (s != LORA_OK) return s;
  }
  if (rope != nullptr) {
    if (rope->rot_dim < 2 || rope->rot_dim > head_dim || rope->rot_dim % 2) return LORA_ERR_SHAPE;
    if ((rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->scale)) return LORA_ERR_ARG;
    if (M > 0 && (rope->positions == nullptr || rope->inv_freq == nullptr)) return LORA_ERR_ARG;
    if ((uintptr_t)rope->positions % 8 || (uintptr_t)rope->inv_freq % 4) return LORA_ERR_SHAPE;
  }
  if (M == 0) return LORA_OK;

  HeadsArgs a{};
  Region in[2] = {}, out[2] = {}, small[4] = {};
  for (int i = 0; i < 2; ++i) {
    const lora_heads_t *h = sets[i];
    if (h == nullptr) continue;
    in[i] = region(h->x, h->ld_row, h->ld_head, D, M, h->n_heads, eb);
    out[i] = region(h->out, h->ldo_row, h->ldo_head, D, M, h->n_heads, eb);
    small[i] = region(h->weight, 0, 0, D, 1, 1, eb);
    a.s[i] = HeadSet{h->x, h->weight, h->out, h->ld_row, h->ld_head, h->ldo_row, h->ldo_head, h->n_heads};
  }
  if (rope != nullptr) {
    small[2] = region(rope->positions, 0, 0, M, 1, 1, 8);
    small[3] = region(rope->inv_freq, 0, 0, rope->rot_dim / 2, 1, 1, 4);
    a.pos = rope->positions;
    a.inv_freq = rope->inv_freq;
    a.rot = rope->rot_dim;
    a.interleaved = rope->interleaved;
    a.scale = rope->scale;
  }
  if (overlap(out[0], out[1])) return LORA_ERR_ARG;
  for (int i = 0; i < 2; ++i) {
    if (sets[i] == nullptr) continue;
    for (int j = 0; j < 2; ++j)
      if (!(i == j && in_place(M, sets[i])) && overlap(out[i], in[j])) return LORA_ERR_ARG;
    for (const Region &r : small)
      if (overlap(out[i], r)) return LORA_ERR_ARG;
  }
  a.dtype = dtype;
  a.M = M;
  a.D = head_dim;
  a.eps = eps;
  return launch_heads(a, (hipStream_t)stream) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // extern "C"
