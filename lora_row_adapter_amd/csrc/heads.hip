// heads.hip -- norm and rotation of query and key heads (include/lora_heads.h).
//
// Bound by memory: every value is read and written once.  A head's columns are
// taken in units of two vectors of E columns, those of the first and of the
// second half that turn together (interleaved, or past the rotated columns,
// two vectors on end), so a lane holds whole pairs and nothing is exchanged but
// the sum of squares, over the 2^n lanes that share a head; a 128-byte line is
// read by eight lanes.  The heads of all rows form one list, of which a
// workgroup takes a run: one token's 72 heads of 128 spread over three
// workgroups, and rows of few heads share one.  A workgroup computes the angles
// of its rows once, for all their heads.
//
// Sums of squares and angles are taken in 64 bits (squares of values past 2^64
// leave fp32's range, and a position times a frequency needs more than 24 bits
// of turns), products in 32.
#include <algorithm>

#include "kernels.hpp"

namespace lora {

namespace {

template <typename T, int E>
struct Vec {
  T v[E];
};
template <typename T, int E>
__device__ __forceinline__ Vec<T, E> load(const T *p) {
  Vec<T, E> r;
  __builtin_memcpy(&r, __builtin_assume_aligned(p, E * sizeof(T)), sizeof(r));
  return r;
}
// (whole vectors past the caches: what is written once is read by another kernel)
template <typename T, int E>
__device__ __forceinline__ void store(T *p, const Vec<T, E> &r) {
  if constexpr (E * sizeof(T) == 16)
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, r), reinterpret_cast<u32x4_t *>(p));
  else
    __builtin_memcpy(__builtin_assume_aligned(p, E * sizeof(T)), &r, sizeof(r));
}
__device__ __forceinline__ float wide(float v) { return v; }
__device__ __forceinline__ float wide(uint16_t v) { return bf16_bits_to_f32(v); }
template <int E>
__device__ __forceinline__ Vec<float, E> narrow(const float (&f)[E], float) {
  Vec<float, E> r;
#pragma unroll
  for (int e = 0; e < E; ++e) r.v[e] = f[e];
  return r;
}
template <int E>
__device__ __forceinline__ Vec<uint16_t, E> narrow(const float (&f)[E], uint16_t) {
  Vec<uint16_t, E> r;
  if constexpr (E == 1) {
    r.v[0] = f32_to_bf16_bits(f[0]);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const uint32_t p = pack_bf16x2(f[e], f[e + 1]);
      r.v[e] = (uint16_t)p;
      r.v[e + 1] = (uint16_t)(p >> 16);
    }
  }
  return r;
}

// cos and sin of pos * freq.  Turns in 64 bits, their fraction in 32.
__device__ __forceinline__ float2 turn(int64_t pos, float freq, float scale) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double t = (double)pos * (double)freq * kInvTwoPi;
  const float f = (float)(t - rint(t));
  float s, c;
  sincospif(2.f * f, &s, &c);
  return make_float2(c * scale, s * scale);
}

// 1 / sqrt(a), a >= 0: the instruction's estimate and two Newton steps.
__device__ __forceinline__ double inverse_root(double a) {
  double r = __builtin_amdgcn_rsq(a);
  if (a > 0 && a < __builtin_inf()) {
#pragma unroll
    for (int i = 0; i < 2; ++i) r = __builtin_fma(0.5 * r, __builtin_fma(-a * r, r, 1.0), r);
  }
  return r;
}

// v from the lane that a DPP control names, of the same 16.
template <int kCtrl>
__device__ __forceinline__ double from(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, kCtrl, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), kCtrl, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over the 2^n lanes that share a head.
__device__ __forceinline__ double over_lanes(double v, int n) {
  if (n > 0) v += from<0xB1>(v);   // lane ^ 1
  if (n > 1) v += from<0x4E>(v);   // lane ^ 2
  if (n > 2) v += from<0x141>(v);  // 7 - lane of eight
  if (n > 3) v += from<0x140>(v);  // 15 - lane of sixteen
  if (n > 4) v += __shfl_xor(v, 16);
  if (n > 5) v += __shfl_xor(v, 32);
  return v;
}

// UPL: units a lane holds (where a head has more than 64).
template <typename T, int E, int UPL>
__global__ __launch_bounds__(256) void k_heads(HeadsArgs a) {
  extern __shared__ float2 cs[];
  const uint32_t H = (uint32_t)(a.s[0].n + a.s[1].n);
  const uint32_t first = blockIdx.x * a.per_block, total = (uint32_t)a.M * H;
  const uint32_t n = min(a.per_block, total - first), row0 = first / H;
  const int half = a.pos ? a.rot >> 1 : 0, rot = 2 * half;
  if (a.pos) {
    const uint32_t pairs = ((first + n - 1) / H - row0 + 1) * (uint32_t)half;
    for (uint32_t i = threadIdx.x; i < pairs; i += 256) {
      const uint32_t r = i / (uint32_t)half, j = i - r * (uint32_t)half;
      const int64_t pos = a.pos[row0 + r];
      if (pos >= 0) cs[i] = turn(pos, a.inv_freq[j], a.scale);
    }
    __syncthreads();
  }

  const uint32_t sub = threadIdx.x & ((1u << a.lanes) - 1), step = 256u >> a.lanes;
  // this lane's units: columns of the two vectors (from D on: none, and column 0
  // is read in their place)
  const int turned = half / E;
  int ca[UPL], cb[UPL];
  Vec<T, E> wa[2][UPL], wb[2][UPL];
#pragma unroll
  for (int q = 0; q < UPL; ++q) {
    const int u = (int)(sub + ((uint32_t)q << a.lanes));
    if (u < turned) {
      ca[q] = a.interleaved ? 2 * E * u : E * u;
      cb[q] = a.interleaved ? ca[q] + E : half + E * u;
    } else {
      ca[q] = rot + 2 * E * (u - turned);
      cb[q] = ca[q] + E;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (a.s[s].w == nullptr) continue;
      wa[s][q] = load<T, E>((const T *)a.s[s].w + (ca[q] < a.D ? ca[q] : 0));
      wb[s][q] = load<T, E>((const T *)a.s[s].w + (cb[q] < a.D ? cb[q] : 0));
    }
  }

  // The heads of this lane's list, the next one's values on their way while one
  // is worked on.
  struct Item {
    Vec<T, E> p[UPL], t[UPL];
    T *y;
    uint32_t row;
    bool second, live;  // of k; not padding
  };
  uint32_t i = threadIdx.x >> a.lanes, row = (first + i) / H, slot = first + i - row * H;
  const uint32_t rows_on = step / H, slots_on = step - rows_on * H, nq = (uint32_t)a.s[0].n;
  auto fetch = [&](Item &it) {
    it.row = row;
    it.second = slot >= nq;
    const HeadSet &hs = a.s[it.second];
    const int64_t h = it.second ? slot - nq : slot;
    const T *x = (const T *)hs.x + row * hs.ldr + h * hs.ldh;
    it.y = (T *)hs.out + row * hs.ldor + h * hs.ldoh;
    it.live = !a.pos || a.pos[row] >= 0;
#pragma unroll
    for (int q = 0; q < UPL; ++q) {
      it.p[q] = load<T, E>(x + (ca[q] < a.D ? ca[q] : 0));
      it.t[q] = load<T, E>(x + (cb[q] < a.D ? cb[q] : 0));
    }
    i += step;
    row += rows_on;
    slot += slots_on;
    if (slot >= H) {
      slot -= H;
      ++row;
    }
  };
  if (i >= n) return;
  Item next;
  fetch(next);
  for (;;) {
    const Item it = next;
    const bool more = i < n;
    if (more) fetch(next);
    float va[UPL][E], vb[UPL][E];
#pragma unroll
    for (int q = 0; q < UPL; ++q)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        va[q][e] = wide(it.p[q].v[e]);
        vb[q][e] = wide(it.t[q].v[e]);
      }
    if (a.s[it.second].w != nullptr) {
      double sum = 0;
#pragma unroll
      for (int q = 0; q < UPL; ++q) {
        double pa = 0, pb = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          pa = __builtin_fma((double)va[q][e], (double)va[q][e], pa);
          pb = __builtin_fma((double)vb[q][e], (double)vb[q][e], pb);
        }
        sum += (ca[q] < a.D ? pa : 0) + (cb[q] < a.D ? pb : 0);
      }
      sum = over_lanes(sum, a.lanes);
      const double r = inverse_root(sum * a.inv_d + (double)a.eps);
      // bf16 has room for a factor rounded to fp32, where that has room for it
      const float rf = (float)r;
      if (sizeof(T) == 2 && r > 0x1p-100 && r < 0x1p100) {
#pragma unroll
        for (int q = 0; q < UPL; ++q)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            va[q][e] *= rf;
            vb[q][e] *= rf;
          }
      } else {
#pragma unroll
        for (int q = 0; q < UPL; ++q)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            va[q][e] = (float)((double)va[q][e] * r);
            vb[q][e] = (float)((double)vb[q][e] * r);
          }
      }
#pragma unroll
      for (int q = 0; q < UPL; ++q)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          va[q][e] *= wide(it.second ? wa[1][q].v[e] : wa[0][q].v[e]);
          vb[q][e] *= wide(it.second ? wb[1][q].v[e] : wb[0][q].v[e]);
        }
    }
    const float2 *c = cs + (it.row - row0) * (uint32_t)half;
#pragma unroll
    for (int q = 0; q < UPL; ++q) {
      const int u = (int)(sub + ((uint32_t)q << a.lanes));
      if (u < turned) {
        float2 w[E];
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = c[E * u + e];
        if (a.interleaved) {
          float f[2 * E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            f[e] = va[q][e];
            f[E + e] = vb[q][e];
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float p = f[2 * e], t = f[2 * e + 1];
            f[2 * e] = p * w[e].x - t * w[e].y;
            f[2 * e + 1] = t * w[e].x + p * w[e].y;
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            va[q][e] = f[e];
            vb[q][e] = f[E + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float p = va[q][e], t = vb[q][e];
            va[q][e] = p * w[e].x - t * w[e].y;
            vb[q][e] = t * w[e].x + p * w[e].y;
          }
        }
      }
      if (it.live) {
        if (ca[q] < a.D) store<T, E>(it.y + ca[q], narrow<E>(va[q], T{}));
        if (cb[q] < a.D) store<T, E>(it.y + cb[q], narrow<E>(vb[q], T{}));
      }
    }
    if (!more) break;
  }
}

template <typename T, int E, int UPL>
void launch(const HeadsArgs &a, uint32_t blocks, size_t lds, hipStream_t st) {
  hipLaunchKernelGGL((k_heads<T, E, UPL>), dim3(blocks), dim3(256), lds, st, a);
}

}  // namespace

hipError_t launch_heads(const HeadsArgs &all, hipStream_t st) {
  const int64_t H = (int64_t)all.s[0].n + all.s[1].n, eb = all.dtype == 1 ? 2 : 4;
  const int half = all.pos ? all.rot / 2 : 0, rot = 2 * half;
  // the widest vectors of up to 16 bytes that all columns, strides and addresses
  // are whole numbers of
  int E = (int)(16 / eb);
  auto fits = [&](int e) {
    if (half % e || (all.D - rot) % e) return false;
    for (const HeadSet &s : all.s) {
      if (s.n == 0) continue;
      if (((uintptr_t)s.x | (uintptr_t)s.out | (uintptr_t)s.w) % (e * eb)) return false;
      if (all.M > 1 && (s.ldr % e || s.ldor % e)) return false;
      if (s.n > 1 && (s.ldh % e || s.ldoh % e)) return false;
    }
    return true;
  };
  while (E > 1 && !fits(E)) E /= 2;
  const int units = half / E + (all.D - rot + 2 * E - 1) / (2 * E);
  int lanes = 0;
  while (lanes < 6 && (1 << lanes) < units) ++lanes;
  const int upl = (units + 63) / 64;
  // items of a workgroup: one round, or as many as leave 1024 workgroups, which
  // the 256 CUs hold at once -- while the angles of all its rows fit 32 KiB of LDS.
  // 8192 rows of 72 heads of 128 in bf16: 18 rounds 67.9 us (4.45 TB/s; a copy
  // makes 4.96), 16 rounds 88 (1152 workgroups), 8 77, 4 71.
  const int64_t round = 256 >> lanes;
  auto bytes = [&](int64_t per) { return (size_t)((per - 1) / H + 2) * half * sizeof(float2); };
  int64_t rounds = std::min<int64_t>(64, (all.M * H + round * 1024 - 1) / (round * 1024));
  while (rounds > 1 && bytes(rounds * round) > 32768) --rounds;

  // rows a launch: a grid of 2^32 threads or more is cut off without an error
  const int64_t slab = std::max<int64_t>(1, std::min<int64_t>(int64_t(1) << 30, (rounds * round) << 22) / H);
  for (int64_t m0 = 0; m0 < all.M; m0 += slab) {
    HeadsArgs a = all;
    a.M = std::min(slab, all.M - m0);
    a.lanes = lanes;
    a.per_block = (uint32_t)(rounds * round);
    a.inv_d = 1.0 / all.D;
    for (HeadSet &s : a.s) {
      if (s.n == 0) continue;
      s.x = (const uint8_t *)s.x + m0 * s.ldr * eb;
      s.out = (uint8_t *)s.out + m0 * s.ldor * eb;
    }
    if (a.pos) a.pos += m0;
    const uint32_t blocks = (uint32_t)((a.M * H + a.per_block - 1) / a.per_block);
    const size_t lds = bytes(a.per_block);
    if (eb == 2) {
      if (E == 8) launch<uint16_t, 8, 1>(a, blocks, lds, st);
      else if (E == 4 && upl == 1) launch<uint16_t, 4, 1>(a, blocks, lds, st);
      else if (E == 4) launch<uint16_t, 4, 2>(a, blocks, lds, st);
      else if (E == 2 && upl == 1) launch<uint16_t, 2, 1>(a, blocks, lds, st);
      else if (E == 2) launch<uint16_t, 2, 4>(a, blocks, lds, st);
      else if (upl == 1) launch<uint16_t, 1, 1>(a, blocks, lds, st);
      else launch<uint16_t, 1, 8>(a, blocks, lds, st);
    } else {
      if (E == 4 && upl == 1) launch<float, 4, 1>(a, blocks, lds, st);
      else if (E == 4) launch<float, 4, 2>(a, blocks, lds, st);
      else if (E == 2 && upl == 1) launch<float, 2, 1>(a, blocks, lds, st);
      else if (E == 2) launch<float, 2, 4>(a, blocks, lds, st);
      else if (upl == 1) launch<float, 1, 1>(a, blocks, lds, st);
      else launch<float, 1, 8>(a, blocks, lds, st);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lora
