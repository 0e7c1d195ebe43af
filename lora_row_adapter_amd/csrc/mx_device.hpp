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

// 16 bytes of a row in registers: kElems consecutive elements, loaded and
// stored as one vector at any alignment of the element size (global memory
// takes unaligned vectors; the row length need not be a multiple).  A block
// of 32 elements is kLanes neighbouring lanes' chunks.
template <typename T>
struct Chunk {
  static constexpr int kElems = 16 / sizeof(T), kLanes = kBlock / kElems;
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
  }
  __device__ __forceinline__ void set2(int i, float lo, float hi) {  // i even
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(lo);
      w[i + 1] = __float_as_uint(hi);
    } else {
      w[i >> 1] = pack_bf16x2(lo, hi);
    }
  }
  // The same values, unknown to the compiler.
  __device__ __forceinline__ void hide() {
    asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  // Chunk c of a row, of which n elements are inside it.
  __device__ __forceinline__ void load(const T *row, int64_t c, int n) {
    const T *p = row + c * kElems;
    if (n == kElems) {
      __builtin_memcpy(w, p, 16);
      return;
    }
    zero();
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kElems; ++i)
        if (i < n) w[i] = __float_as_uint(p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kElems; ++i)
        if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  // Non-temporal: lines that nothing reads again in this kernel.  9216 x 8192
  // fp32 values read back from fp4 codes take 48 us this way, 75 with plain
  // stores; 8192 x 4096 bf16 from fp8 15.8 and 19.5.
  __device__ __forceinline__ void store(T *row, int64_t c, int n) const {
    typedef uint32_t Vec __attribute__((ext_vector_type(4), aligned(2)));
    T *p = row + c * kElems;
    if (n == kElems) {
      __builtin_nontemporal_store((Vec){w[0], w[1], w[2], w[3]}, (Vec *)p);
      return;
    }
#pragma unroll
    for (int i = 0; i < kElems; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 4) p[i] = __uint_as_float(w[i]);
        else p[i] = (T)(w[i >> 1] >> (16 * (i & 1)));
      }
  }
  // elements of chunk c inside a row of k
  static __device__ __forceinline__ int len(int64_t c, int64_t k) {
    const int64_t left = k - c * kElems;
    return left >= kElems ? kElems : left > 0 ? (int)left : 0;
  }
};

// max over LANES neighbouring lanes (4 or 8).  DPP moves: no LDS traffic.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
  v = v > o ? v : o;
  if constexpr (LANES == 8) {
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);  // lanes 7 6 .. 0
    v = v > o ? v : o;
  }
  return v;
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

// Values (already divided by their scale, finite) to codes.  The conversions
// round to nearest even; E2M1's saturates by itself, E4M3's makes NaNs past
// 448, so it gets clamped values.  (Checked on the device against the tables
// for every bf16 pattern and 10^6 fp32 ones.)
__device__ __forceinline__ uint32_t codes4_fp8(const float *v) {
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i], 448.f, -448.f);
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], r, true);
}
__device__ __forceinline__ uint32_t codes4_fp4(const float *v) {  // in the lower 16 bits
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], 1.0f, 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
}

// Quantise a block: this lane's N values (zeros past the row's end), chunk c
// of the row; writes codes and (the block's first lane) the scale.  All lanes
// of a block call it together.
template <int FMT, int N>
__device__ __forceinline__ void quantise_chunk(const float (&v)[N], int64_t c, bool live,
                                               uint8_t *qrow, uint8_t *srow) {
  constexpr int LANES = kBlock / N;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  top = lanes_max<LANES>(top);
  const uint32_t s = scale_byte<FMT>(top);
  float u[N];
  const float inv = inv_scale(s > 252u ? 252u : s);
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = s == 255u ? 0.f : v[i] * inv;
  if (!live) return;
  if constexpr (FMT == kFp8) {
    uint32_t *q = reinterpret_cast<uint32_t *>(qrow + c * N);
    if constexpr (N == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(codes4_fp8(u), codes4_fp8(u + 4));
    else *q = codes4_fp8(u);
  } else {
    uint8_t *q = qrow + c * (N / 2);
    if constexpr (N == 8) *reinterpret_cast<uint32_t *>(q) = codes4_fp4(u) | (codes4_fp4(u + 4) << 16);
    else *reinterpret_cast<uint16_t *>(q) = (uint16_t)codes4_fp4(u);
  }
  if ((threadIdx.x & (LANES - 1)) == 0) srow[c / LANES] = (uint8_t)s;
}

}  // namespace mx
}  // namespace lora
