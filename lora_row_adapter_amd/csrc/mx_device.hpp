// mx_device.hpp -- device helpers of the microscaled formats (32 elements per
// power-of-two scale; include/lora_mx.h).  Internal.
#pragma once

#include "kernels.hpp"

namespace lora {
namespace mx {

constexpr int kFp8 = LORA_MX_FP8, kFp4 = LORA_MX_FP4;
constexpr int kBlock = 32;

// Bytes of one block's codes.
__host__ __device__ constexpr int block_bytes(int fmt) { return fmt == kFp8 ? 32 : 16; }

// Eight consecutive elements of a row in registers, loaded and stored as
// whole 16-byte vectors at any alignment of the element size (global memory
// takes unaligned vectors; the row length need not be a multiple of 8).
template <typename T>
struct Chunk;

template <>
struct Chunk<uint16_t> {  // bf16
  uint32_t w[4];
  __device__ __forceinline__ void load(const uint16_t *p) { __builtin_memcpy(w, p, 16); }
  __device__ __forceinline__ void store(uint16_t *p) const { __builtin_memcpy(p, w, 16); }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
  }
  __device__ __forceinline__ void set2(int i, float lo, float hi) { w[i >> 1] = pack_bf16x2(lo, hi); }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  // elements [0, n) only (n < 8)
  __device__ __forceinline__ void load_part(const uint16_t *p, int n) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[2 * i] | (v[2 * i + 1] << 16);
  }
  __device__ __forceinline__ void store_part(uint16_t *p, int n) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
};

template <>
struct Chunk<float> {
  float w[8];
  __device__ __forceinline__ void load(const float *p) { __builtin_memcpy(w, p, 32); }
  __device__ __forceinline__ void store(float *p) const { __builtin_memcpy(p, w, 32); }
  __device__ __forceinline__ float get(int i) const { return w[i]; }
  __device__ __forceinline__ void set2(int i, float lo, float hi) {
    w[i] = lo;
    w[i + 1] = hi;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.f;
  }
  __device__ __forceinline__ void load_part(const float *p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? p[i] : 0.f;
  }
  __device__ __forceinline__ void store_part(float *p, int n) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = w[i];
  }
};

// Elements of chunk `c` of a row of k: 8 inside, fewer at the end, 0 past it.
__device__ __forceinline__ int chunk_len(int64_t c, int64_t k) {
  const int64_t left = k - c * 8;
  return left >= 8 ? 8 : left > 0 ? (int)left : 0;
}

template <typename T>
__device__ __forceinline__ void load_chunk(Chunk<T> &v, const T *row, int64_t c, int n) {
  if (n == 8) v.load(row + c * 8);
  else if (n > 0) v.load_part(row + c * 8, n);
  else v.zero();
}
template <typename T>
__device__ __forceinline__ void store_chunk(const Chunk<T> &v, T *row, int64_t c, int n) {
  if (n == 8) v.store(row + c * 8);
  else if (n > 0) v.store_part(row + c * 8, n);
}

// max over the four lanes of a quad (the four chunks of one block).  DPP
// quad_perm moves: no LDS traffic.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
  return v > o ? v : o;
}

// Scale byte of a block whose largest magnitude has the fp32 bits `top`: the
// biased exponent less the exponent of the format's largest code, not below
// 0 (so subnormal and zero blocks take 2^-127); 255 for infinities and NaNs.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  constexpr int emax = FMT == kFp8 ? 8 : 2;
  const int e = (int)(top >> 23);
  return e == 255 ? 255u : (uint32_t)(e > emax ? e - emax : 0);
}
// 1 / scale, exact: 2^(127 - s) for s <= 252 (what scale_byte gives for
// finite blocks).
__device__ __forceinline__ float inv_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }
// 2^(s - 127): 2^-127 is the subnormal 0x00400000; 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// Eight values (already divided by their scale, finite) to codes.  The
// conversions round to nearest even; E2M1's saturates by itself, E4M3's
// makes NaNs past 448, so it gets clamped values.  (Checked on the device
// against the tables for every bf16 pattern and 10^6 fp32 ones.)
__device__ __forceinline__ uint32_t codes_fp4(const float (&v)[8]) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
  return r;
}
__device__ __forceinline__ uint2 codes_fp8(const float (&v)[8]) {
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i], 448.f, -448.f);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Quantise the quad's block: this lane's eight values (zeros past the row's
// end), chunk `c` of the row; writes codes and (first lane) the scale.  All
// four lanes of a quad call it together.
template <int FMT>
__device__ __forceinline__ void quantise_chunk(const float (&v)[8], int64_t c, bool live,
                                               uint8_t *qrow, uint8_t *srow) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  top = quad_max(top);
  const uint32_t s = scale_byte<FMT>(top);
  float u[8];
  const float inv = inv_scale(s > 252u ? 252u : s);
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = s == 255u ? 0.f : v[i] * inv;
  if (!live) return;
  if constexpr (FMT == kFp8)
    *reinterpret_cast<uint2 *>(qrow + c * 8) = codes_fp8(u);
  else
    *reinterpret_cast<uint32_t *>(qrow + c * 4) = codes_fp4(u);
  if ((threadIdx.x & 3) == 0) srow[c >> 2] = (uint8_t)s;
}

}  // namespace mx
}  // namespace lora
