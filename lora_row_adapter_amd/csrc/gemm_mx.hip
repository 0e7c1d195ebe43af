// gemm_mx.hip -- base projection on microscaled operands (include/lora_mx.h):
//   y[m, n] = sum_b 2^(sx[m,b] - 127) 2^(sw[n,b] - 127) sum_{i < 32} cx[m,32b+i] cw[n,32b+i]
// with x in fp8 or fp4 and W in fp4, on gfx950's scaled matrix instruction
// 16x16x128, which takes both operands' codes and a scale byte per row and
// 32 elements, and accumulates in fp32.
//
// Operand layout of the instruction (checked on the device against the
// definition with random codes and scales; g = lane / 16):
//   scale: lane's byte is that of row lane % 16 and block g of the four
//   fp4:   lane holds block g of its row (16 bytes)
//   fp8:   registers 0-3 hold bytes 16g .. 16g+15 of the row's 128, registers
//          4-7 bytes 64+16g .. 64+16g+15: halves of blocks g/2 and 2 + g/2
// Which four blocks of a row one instruction multiplies is free as long as
// both operands and the scales agree.
#include "mx_device.hpp"

namespace lora {

using namespace mx;

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr uint32_t kOob = 0xFFFFFFF0u;  // past every buffer: loads give zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, 0x00020000);
}
__device__ __forceinline__ i32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ uint32_t load4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}

__device__ __forceinline__ i32x8_t frag4(i32x4_t v) {
  return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
}
__device__ __forceinline__ i32x8_t frag8(i32x4_t a, i32x4_t b) {
  return i32x8_t{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// acc += W fragment (fp4, rows of the result) x x fragment (columns)
template <int XF, int J>
__device__ __forceinline__ f32x4_t mfma(i32x8_t w, i32x8_t x, f32x4_t acc, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, XF == kFp8 ? 0 : 4, J,
                                                          (int)sw, J, (int)sx);
}

// Scale bytes of the blocks from `first` on that exist (first + byte < nb);
// the others become 0: they meet zero codes, and no stray 255 makes a NaN.
__device__ __forceinline__ uint32_t keep_scales(uint32_t s, int first, int nb) {
  const int n = nb - first;
  return n >= 4 ? s : n <= 0 ? 0u : s & ((1u << (8 * n)) - 1u);
}

// Four waves split k of one tile of 16 W rows x 16 MF rows of x; each step is
// 16 blocks (512 elements): lane g of a row takes the 64 (fp4) contiguous
// bytes of blocks 4g .. 4g+3, one per instruction, and their four scales in
// one load.  The waves' sums meet in LDS.
template <int XF, int MF>
__global__ __launch_bounds__(256) void k_gemm_mx_rows(MxGemmArgs p) {
  __shared__ f32x4_t red[4][MF][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int tm = blockIdx.x % p.tiles_m, tn = blockIdx.x / p.tiles_m;
  const int m0 = tm * 16 * MF, n0 = tn * 16;
  const int mr = min(16 * MF, p.M - m0), nr = min(16, p.N - n0);
  const auto rw = rsrc(p.w + (int64_t)n0 * p.ldw, (uint32_t)(nr * p.ldw));
  const auto rws = rsrc(p.wsc + (int64_t)n0 * p.ldws, (uint32_t)(nr * p.ldws));
  const auto rx = rsrc(p.x + (int64_t)m0 * p.ldx, (uint32_t)(mr * p.ldx));
  const auto rxs = rsrc(p.xs + (int64_t)m0 * p.ldxs, (uint32_t)(mr * p.ldxs));

  f32x4_t acc[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  for (int b0 = wave * 16; b0 < p.nb; b0 += 64) {
    // offsets of block b0 + 4g + j; past the row's end: nothing
    auto at = [&](int row, int64_t ld, int b, int bytes, int add) {
      return b < p.nb ? (uint32_t)(row * ld + (int64_t)b * bytes + add) : kOob;
    };
    i32x4_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = load16(rw, at(r, p.ldw, b0 + 4 * g + j, 16, 0));
    const int sb = b0 + 4 * g;
    const uint32_t sw = keep_scales(load4(rws, sb < p.nb ? (uint32_t)(r * p.ldws + sb) : kOob), sb, p.nb);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int row = r + 16 * i;
      const uint32_t sx = keep_scales(load4(rxs, sb < p.nb ? (uint32_t)(row * p.ldxs + sb) : kOob), sb, p.nb);
      i32x8_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (XF == kFp8)
          x[j] = frag8(load16(rx, at(row, p.ldx, b0 + 4 * (g >> 1) + j, 32, (g & 1) * 16)),
                       load16(rx, at(row, p.ldx, b0 + 4 * (2 + (g >> 1)) + j, 32, (g & 1) * 16)));
        else
          x[j] = frag4(load16(rx, at(row, p.ldx, b0 + 4 * g + j, 16, 0)));
      }
      acc[i] = mfma<XF, 0>(frag4(w[0]), x[0], acc[i], sw, sx);
      acc[i] = mfma<XF, 1>(frag4(w[1]), x[1], acc[i], sw, sx);
      acc[i] = mfma<XF, 2>(frag4(w[2]), x[2], acc[i], sw, sx);
      acc[i] = mfma<XF, 3>(frag4(w[3]), x[3], acc[i], sw, sx);
    }
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MF; i += 4) {
    const f32x4_t v = ((red[0][i][lane] + red[1][i][lane]) + red[2][i][lane]) + red[3][i][lane];
    const int m = m0 + 16 * i + r, n = n0 + 4 * g;
    if (m >= p.M) continue;
    uint16_t *dst = p.y + (int64_t)m * p.ldy + n;
    const uint32_t o[2] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    if (n + 4 <= p.N) {
      __builtin_memcpy(dst, o, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) dst[e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
    }
  }
}

template <int XF, int MF>
void launch_rows(MxGemmArgs a, hipStream_t st) {
  a.tiles_m = (a.M + 16 * MF - 1) / (16 * MF);
  a.tiles_n = (a.N + 15) / 16;
  hipLaunchKernelGGL((k_gemm_mx_rows<XF, MF>), dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(256),
                     0, st, a);
}

template <int XF>
void launch_fmt(const MxGemmArgs &a, hipStream_t st) {
  if (a.M <= 16) launch_rows<XF, 1>(a, st);
  else if (a.M <= 32) launch_rows<XF, 2>(a, st);
  else launch_rows<XF, 4>(a, st);
}

}  // namespace

hipError_t launch_gemm_mx(const MxGemmArgs &a, hipStream_t st) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  if (a.xfmt == kFp8) launch_fmt<kFp8>(a, st);
  else launch_fmt<kFp4>(a, st);
  return hipGetLastError();
}

}  // namespace lora
