// heads.hip -- norm and rotation of query and key heads (include/lora_heads.h).
//
// Sums of squares and angles are taken in 64 bits (squares of values past
// 2^64 leave fp32's range, and a position times a frequency needs more than
// 24 bits of turns), products in 32.
#include <algorithm>

#include "kernels.hpp"

namespace lora {

namespace {

constexpr int kMaxD = 1024;

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = f32_to_bf16_bits(v); }

// cos and sin of pos * freq.  Turns in 64 bits, their fraction in 32.
__device__ __forceinline__ float2 turn(int64_t pos, float freq, float scale) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double t = (double)pos * (double)freq * kInvTwoPi;
  const float f = (float)(t - rint(t));
  float s, c;
  sincospif(2.f * f, &s, &c);
  return make_float2(c * scale, s * scale);
}

// One workgroup a row, its four waves every fourth head.
template <typename T>
__global__ __launch_bounds__(256) void k_heads(HeadsArgs a) {
  __shared__ float2 cs[kMaxD / 2];
  __shared__ float u[4][kMaxD];
  const int64_t m = blockIdx.x;
  const int half = a.pos ? a.rot / 2 : 0;
  if (a.pos) {
    const int64_t pos = a.pos[m];
    if (pos < 0) return;
    for (int i = threadIdx.x; i < half; i += 256) cs[i] = turn(pos, a.inv_freq[i], a.scale);
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float *v = u[wave];
  for (int q = 0; q < 2; ++q) {
    const HeadSet &s = a.s[q];
    for (int h = wave; h < s.n; h += 4) {
      const T *x = (const T *)s.x + m * s.ldr + h * s.ldh;
      T *y = (T *)s.out + m * s.ldor + h * s.ldoh;
      double sum = 0;
      for (int j = lane; j < a.D; j += 64) {
        v[j] = load1(x + j);
        sum += (double)v[j] * (double)v[j];
      }
      if (s.w) {
        for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
        const double r = 1.0 / sqrt(sum / a.D + (double)a.eps);
        for (int j = lane; j < a.D; j += 64) v[j] = (float)((double)v[j] * r) * load1((const T *)s.w + j);
      }
      __builtin_amdgcn_wave_barrier();
      for (int i = lane; i < half; i += 64) {
        const int ja = a.interleaved ? 2 * i : i, jb = a.interleaved ? 2 * i + 1 : i + half;
        const float p = v[ja], t = v[jb];
        const float2 w = cs[i];
        store1(y + ja, p * w.x - t * w.y);
        store1(y + jb, t * w.x + p * w.y);
      }
      for (int j = 2 * half + lane; j < a.D; j += 64) store1(y + j, v[j]);
      __builtin_amdgcn_wave_barrier();
    }
  }
}

}  // namespace

hipError_t launch_heads(const HeadsArgs &all, hipStream_t st) {
  constexpr int64_t kSlab = int64_t(1) << 30;
  for (int64_t m0 = 0; m0 < all.M; m0 += kSlab) {
    HeadsArgs a = all;
    a.M = std::min(kSlab, all.M - m0);
    const int64_t eb = a.dtype == 1 ? 2 : 4;
    for (HeadSet &s : a.s) {
      if (s.n == 0) continue;
      s.x = (const uint8_t *)s.x + m0 * s.ldr * eb;
      s.out = (uint8_t *)s.out + m0 * s.ldor * eb;
    }
    if (a.pos) a.pos += m0;
    if (a.dtype == 1) hipLaunchKernelGGL(k_heads<uint16_t>, dim3((unsigned)a.M), dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_heads<float>, dim3((unsigned)a.M), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lora
