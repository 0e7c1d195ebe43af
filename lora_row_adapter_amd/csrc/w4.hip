// w4.hip -- the 4-bit base weight of include/lora_w4.h: laying it out, reading
// it back, and the product
//   y[m, n] = sum_g s[n, g] (sum_{j in g} x[m, j] q[n, j] - z[n, g] sum_{j in g} x[m, j])
//
// A code needs one mask and one OR to be a bf16 number: 0x4300 | q is 128 + q
// exactly, so the matrix instruction multiplies x with 128 + q and, against a
// column of ones, gives the group's sum of x; then
//   tot += s (acc - (128 + z) X)
// in fp32: no weight is rounded.  acc and (128 + z) X are about 143 / 4.6
// times what is left of them (codes are 4.6 off their zero point, root mean
// square), which costs the sum 5 of fp32's 24 bits; y keeps 8.
#include <algorithm>

#include "kernels.hpp"

namespace lora {

namespace {

__device__ __forceinline__ float scale_of(uint32_t w) { return __uint_as_float(w & ~31u); }

// 128 + codes of one dword as the matrix instruction's eight bf16.
__device__ __forceinline__ bf16x8_t codes128(uint32_t w) {
  u32x4_t v;
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = ((w >> (4 * p)) & 0x000F000Fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8_t, v);
}

// ---------------------------------------------------------------- layout
// One workgroup a record: 256 threads a dword of codes each, then its scales.
__global__ __launch_bounds__(256) void k_w4_pack(W4Args a) {
  const int64_t rec = blockIdx.x, tile = rec / a.nb, blk = rec - tile * a.nb;
  uint32_t *out = reinterpret_cast<uint32_t *>(a.w + rec * w4_record(a.sg));
  const int t = threadIdx.x, lane = t >> 2, i = t & 3;
  const int64_t n = tile * 16 + (lane & 15);
  const int64_t j0 = blk * 128 + 32 * i + 8 * (lane >> 4);
  uint32_t w = 0;
  if (n < a.d) {
    const uint8_t *row = a.q + n * a.ldq;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int64_t j = j0 + 2 * p;
      if (j < a.k) {
        const uint32_t b = row[j >> 1];
        w |= (b & 15u) << (4 * p) | (b >> 4) << (16 + 4 * p);
      }
    }
  }
  out[t] = w;
  if (t < 16 * a.sg) {
    const int64_t r = tile * 16 + (t & 15);
    const int64_t g = (blk * 128 + (int64_t)(t >> 4) * (128 / a.sg)) / a.group;
    uint32_t s = 0;
    if (r < a.d && g * a.group < a.k) {
      uint32_t bits = a.scale_dtype == 1
                          ? (uint32_t)((const uint16_t *)a.scales)[r * a.lds + g] << 16
                          : ((const uint32_t *)a.scales)[r * a.lds + g];
      // to 19 significant bits, ties to even; a NaN stays one
      if ((bits & 0x7FFFFFFFu) > 0x7F800000u) bits |= 0x00400000u;
      else bits += 15u + ((bits >> 5) & 1u);
      const uint32_t z = a.zeros ? a.zeros[r * a.ldz + g] & 31u : 8u;
      s = (bits & ~31u) | z;
    }
    out[256 + t] = s;
  }
}

// One workgroup a record, a dword of codes (eight columns of a row) a thread;
// sixteen threads cover a row's 128 columns.
template <typename T>
__global__ __launch_bounds__(256) void k_w4_dequantize(W4Args a) {
  const int64_t rec = blockIdx.x, tile = rec / a.nb, blk = rec - tile * a.nb;
  const uint32_t *in = reinterpret_cast<const uint32_t *>(a.w + rec * w4_record(a.sg));
  const int t = threadIdx.x, row = t >> 4, i = (t >> 2) & 3, h = t & 3;
  const int64_t n = tile * 16 + row, j0 = blk * 128 + 32 * i + 8 * h;
  if (n >= a.d || j0 >= a.k) return;
  const uint32_t w = in[(h * 16 + row) * 4 + i];
  const uint32_t sw = in[256 + (i * a.sg >> 2) * 16 + row];
  const float s = scale_of(sw);
  const int z = (int)(sw & 31u);
  // 19 bits by 5: the products are exact
  float v[8];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    v[2 * p] = s * (float)((int)((w >> (4 * p)) & 15u) - z);
    v[2 * p + 1] = s * (float)((int)((w >> (16 + 4 * p)) & 15u) - z);
  }
  T *y = (T *)a.y + n * a.ldy + j0;
  const int left = (int)min((int64_t)8, a.k - j0);
  T o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (sizeof(T) == 2) o[e] = f32_to_bf16_bits(v[e]);
    else o[e] = v[e];
  }
  if (left == 8 && ((uintptr_t)y & 15) == 0) {
#pragma unroll
    for (int c = 0; c < (int)sizeof(T) / 2; ++c)
      reinterpret_cast<uint4 *>(y)[c] = reinterpret_cast<const uint4 *>(o)[c];
  } else {
    for (int e = 0; e < left; ++e) y[e] = o[e];
  }
}

// ---------------------------------------------------------------- product
// A workgroup takes 16 rows of x and 16 of W, its four waves every fourth
// record of k.
template <int SG>
__global__ __launch_bounds__(256) void k_w4_rows(W4GemmArgs p) {
  __shared__ f32x4_t part[3][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const uint16_t *x = p.x + (int64_t)min(m0 + (lane & 15), p.M - 1) * p.ldx;
  const uint8_t *w = p.w + (int64_t)blockIdx.x * p.nb * w4_record(SG);
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
  f32x4_t tot = {0.f, 0.f, 0.f, 0.f};
  for (int blk = wave; blk < p.nb; blk += 4) {
    const uint8_t *rec = w + (int64_t)blk * w4_record(SG);
    const u32x4_t c = reinterpret_cast<const u32x4_t *>(rec)[lane];
    const uint32_t *sc = reinterpret_cast<const uint32_t *>(rec + kW4Codes) + (lane & 15);
#pragma unroll
    for (int g = 0; g < SG; ++g) {
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f}, sum = acc;
#pragma unroll
      for (int i = g * 4 / SG; i < (g + 1) * 4 / SG; ++i) {
        const int j = blk * 128 + 32 * i + 8 * h;
        u32x4_t xv = {0, 0, 0, 0};
        if (j < p.K) xv = *reinterpret_cast<const u32x4_t *>(x + j);
        const bf16x8_t xf = __builtin_bit_cast(bf16x8_t, xv);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, codes128(c[i]), acc, 0, 0, 0);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, ones, sum, 0, 0, 0);
      }
      const uint32_t sw = sc[g * 16];
      const float s = scale_of(sw), z = (float)(128 + (int)(sw & 31u));
#pragma unroll
      for (int e = 0; e < 4; ++e) tot[e] += s * (acc[e] - z * sum[e]);
    }
  }
  if (wave > 0) part[wave - 1][lane] = tot;
  __syncthreads();
  if (wave > 0) return;
  for (int v = 0; v < 3; ++v) tot += part[v][lane];
  const int n = n0 + (lane & 15);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int m = m0 + 4 * h + e;
    if (m < p.M && n < p.N) p.y[(int64_t)m * p.ldy + n] = f32_to_bf16_bits(tot[e]);
  }
}

}  // namespace

hipError_t launch_w4_pack(const W4Args &a, hipStream_t st) {
  const int64_t recs = (a.d + 15) / 16 * a.nb;
  hipLaunchKernelGGL(k_w4_pack, dim3((unsigned)recs), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_w4_dequantize(const W4Args &a, hipStream_t st) {
  const int64_t recs = (a.d + 15) / 16 * a.nb;
  if (a.dtype == 1)
    hipLaunchKernelGGL(k_w4_dequantize<uint16_t>, dim3((unsigned)recs), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(k_w4_dequantize<float>, dim3((unsigned)recs), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_gemm_w4(const W4GemmArgs &all, hipStream_t st) {
  constexpr int64_t kSlab = 16 * 65535;  // rows a launch
  for (int64_t m0 = 0; m0 < all.M; m0 += kSlab) {
    W4GemmArgs a = all;
    a.M = (int32_t)std::min(kSlab, all.M - m0);
    a.x += m0 * a.ldx;
    a.y += m0 * a.ldy;
    const dim3 grid((a.N + 15) / 16, (a.M + 15) / 16);
    if (a.sg == 1) hipLaunchKernelGGL(k_w4_rows<1>, grid, dim3(256), 0, st, a);
    else if (a.sg == 2) hipLaunchKernelGGL(k_w4_rows<2>, grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_w4_rows<4>, grid, dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lora
