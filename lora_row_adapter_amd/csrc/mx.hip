// mx.hip -- microscaled quantising and reading back, and the root-mean-square
// norm with a microscaled output (include/lora_mx.h).
//
// All three are one pass over the data and bound by its bytes.  A row is cut
// into chunks of eight elements, one lane each, so a block of 32 is a quad of
// lanes: its largest magnitude takes two DPP moves, and a wave's loads and
// stores are contiguous runs of 16 bytes a lane.
#include <algorithm>

#include "mx_device.hpp"

namespace lora {

using namespace mx;

namespace {

constexpr int kThreads = 256;

// A workgroup covers `ty` rows x `tx` chunk columns (tx a power of two, ty *
// tx = 256) in each of UNR steps along the row; blockIdx.x runs over column
// segments first.
struct RowGrid {
  int32_t log_tx;
  uint32_t nseg;    // column segments per row group
  int64_t chunks;   // chunks per row: ceil(k / 32) * 4
};

template <typename T, int FMT, int UNR>
__global__ __launch_bounds__(kThreads) void k_mx_quantize(const T *x, int64_t ldx, int64_t M,
                                                          int64_t k, RowGrid g, uint8_t *q,
                                                          int64_t ldq, uint8_t *sc, int64_t lds) {
  const int tx = 1 << g.log_tx;
  const int lx = threadIdx.x & (tx - 1);
  const uint32_t grp = blockIdx.x / g.nseg, seg = blockIdx.x - grp * g.nseg;
  const int64_t m = (int64_t)grp * (kThreads >> g.log_tx) + (threadIdx.x >> g.log_tx);
  if (m >= M) return;  // whole quads leave: tx >= 4
  const int64_t c0 = (int64_t)seg * (UNR << g.log_tx) + lx;
  const T *row = x + m * ldx;
  Chunk<T> v[UNR];
#pragma unroll
  for (int i = 0; i < UNR; ++i) {
    const int64_t c = c0 + ((int64_t)i << g.log_tx);
    load_chunk(v[i], row, c, chunk_len(c, k));
  }
#pragma unroll
  for (int i = 0; i < UNR; ++i) {
    const int64_t c = c0 + ((int64_t)i << g.log_tx);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[i].get(e);
    quantise_chunk<FMT>(f, c, c < g.chunks, q + m * ldq, sc + m * lds);
  }
}

template <typename T, int FMT, int UNR>
__global__ __launch_bounds__(kThreads) void k_mx_dequantize(const uint8_t *q, int64_t ldq,
                                                            const uint8_t *sc, int64_t lds,
                                                            int64_t M, int64_t k, RowGrid g, T *y,
                                                            int64_t ldy) {
  const int tx = 1 << g.log_tx;
  const int lx = threadIdx.x & (tx - 1);
  const uint32_t grp = blockIdx.x / g.nseg, seg = blockIdx.x - grp * g.nseg;
  const int64_t m = (int64_t)grp * (kThreads >> g.log_tx) + (threadIdx.x >> g.log_tx);
  if (m >= M) return;
  const int64_t c0 = (int64_t)seg * (UNR << g.log_tx) + lx;
  const uint8_t *qrow = q + m * ldq, *srow = sc + m * lds;
  uint2 w[UNR];
  uint32_t s[UNR];
#pragma unroll
  for (int i = 0; i < UNR; ++i) {
    const int64_t c = c0 + ((int64_t)i << g.log_tx);
    const bool live = c < g.chunks;
    w[i] = make_uint2(0, 0);
    s[i] = 0;
    if (live) {
      if constexpr (FMT == kFp8) w[i] = *reinterpret_cast<const uint2 *>(qrow + c * 8);
      else w[i].x = *reinterpret_cast<const uint32_t *>(qrow + c * 4);
      s[i] = srow[c >> 2];
    }
  }
#pragma unroll
  for (int i = 0; i < UNR; ++i) {
    const int64_t c = c0 + ((int64_t)i << g.log_tx);
    const float f = scale_value(s[i]);
    Chunk<T> o;
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    if constexpr (FMT == kFp8) {
      const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].x, false);
      const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].x, true);
      const f32x2_t d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].y, false);
      const f32x2_t e = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].y, true);
      o.set2(0, a[0] * f, a[1] * f);
      o.set2(2, b[0] * f, b[1] * f);
      o.set2(4, d[0] * f, d[1] * f);
      o.set2(6, e[0] * f, e[1] * f);
    } else {
      const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i].x, 1.0f, 0);
      const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i].x, 1.0f, 1);
      const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i].x, 1.0f, 2);
      const f32x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i].x, 1.0f, 3);
      o.set2(0, a[0] * f, a[1] * f);
      o.set2(2, b[0] * f, b[1] * f);
      o.set2(4, d[0] * f, d[1] * f);
      o.set2(6, e[0] * f, e[1] * f);
    }
    store_chunk(o, y + m * ldy, c, chunk_len(c, k));
  }
}

// v rounded to fp32 "to odd": toward zero, with the last bit set when that
// was inexact.  A further rounding of the result to fewer bits than fp32
// minus two is then the correct rounding of v itself, so bf16 and the 8- and
// 4-bit codes are each rounded once from the 64-bit value.
__device__ __forceinline__ float to_odd(double v) {
  const float f = (float)v;
  const double d = (double)f;
  uint32_t b = __float_as_uint(f);
  if (d != v && !(b & 1u)) b += fabs(d) > fabs(v) ? 0xffffffffu : 1u;
  return __uint_as_float(b);
}

template <typename T>
__device__ __forceinline__ float to_out(double v) {
  if constexpr (sizeof(T) == 4) return (float)v;
  else return to_odd(v);  // rounded to bf16 where it is packed
}

struct NormArgs {
  const void *x, *res, *w;
  void *h, *y;
  uint8_t *q, *sc;
  int64_t ldx, ldr, ldh, ldy, ldq, lds;
  int64_t M, k, chunks;
  double eps, inv_k;
  int32_t log_tpr;  // threads per row (a power of two, 4 .. 1024)
};

// Sum over the threads of a row (1 << log_tpr of them, aligned).
__device__ __forceinline__ double row_sum(double s, int log_tpr, double *red) {
  const int in_wave = log_tpr < 6 ? log_tpr : 6;
  for (int i = 0; i < in_wave; ++i) s += __shfl_xor(s, 1 << i, 64);
  if (log_tpr > 6) {  // one row per workgroup
    const int nw = 1 << (log_tpr - 6);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0;
    for (int i = 0; i < nw; ++i) s += red[i];
  }
  return s;
}

// One row per 1 << log_tpr threads.  C > 0: each thread keeps its C chunks of
// x and the residual in registers, so every input is read once; C == 0: rows
// too long for that are read twice.
template <typename T, int FMT, int C>
__global__ __launch_bounds__(1024) void k_rmsnorm(NormArgs a) {
  __shared__ double red[16];
  const int tpr = 1 << a.log_tpr;
  const int lx = threadIdx.x & (tpr - 1);
  const int64_t m = (int64_t)blockIdx.x * (blockDim.x >> a.log_tpr) + (threadIdx.x >> a.log_tpr);
  if (m >= a.M) return;  // whole rows leave; rows of several waves are alone in their workgroup
  const T *x = (const T *)a.x + m * a.ldx;
  const T *r = a.res ? (const T *)a.res + m * a.ldr : nullptr;
  const T *w = (const T *)a.w;
  T *h = a.h ? (T *)a.h + m * a.ldh : nullptr;
  T *y = a.y ? (T *)a.y + m * a.ldy : nullptr;
  uint8_t *q = FMT ? a.q + m * a.ldq : nullptr;
  uint8_t *sc = FMT ? a.sc + m * a.lds : nullptr;

  auto finish = [&](const Chunk<T> &xv, const Chunk<T> &rv, int64_t c, int n, double rstd) {
    Chunk<T> wv, o;
    load_chunk(wv, w, c, n);
    float f[8];
    double hv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) hv[e] = (double)xv.get(e) + (double)rv.get(e);
    if (h != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) o.set2(e, to_out<T>(hv[e]), to_out<T>(hv[e + 1]));
      store_chunk(o, h, c, n);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) hv[e] = hv[e] * rstd * (double)wv.get(e);
    if (sizeof(T) == 4 && y != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) o.set2(e, (float)hv[e], (float)hv[e + 1]);
      store_chunk(o, y, c, n);
    }
    if (FMT || sizeof(T) == 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = to_odd(hv[e]);
    }
    if (sizeof(T) == 2 && y != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) o.set2(e, f[e], f[e + 1]);
      store_chunk(o, y, c, n);
    }
    if constexpr (FMT != 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = e < n ? f[e] : 0.f;  // 0 * inf past the row's end
      quantise_chunk<FMT>(f, c, c < a.chunks, q, sc);
    }
  };

  double s = 0;
  if constexpr (C > 0) {
    Chunk<T> xv[C], rv[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int64_t c = ((int64_t)i << a.log_tpr) + lx;
      const int n = chunk_len(c, a.k);
      load_chunk(xv[i], x, c, n);
      if (r) load_chunk(rv[i], r, c, n);
      else rv[i].zero();
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double v = (double)xv[i].get(e) + (double)rv[i].get(e);
        s = fma(v, v, s);
      }
    s = row_sum(s, a.log_tpr, red);
    const double rstd = 1.0 / sqrt(s * a.inv_k + a.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int64_t c = ((int64_t)i << a.log_tpr) + lx;
      if (c < a.chunks) finish(xv[i], rv[i], c, chunk_len(c, a.k), rstd);
    }
  } else {
    for (int64_t c = lx; c < a.chunks; c += tpr) {
      Chunk<T> xv, rv;
      const int n = chunk_len(c, a.k);
      load_chunk(xv, x, c, n);
      if (r) load_chunk(rv, r, c, n);
      else rv.zero();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double v = (double)xv.get(e) + (double)rv.get(e);
        s = fma(v, v, s);
      }
    }
    s = row_sum(s, a.log_tpr, red);
    const double rstd = 1.0 / sqrt(s * a.inv_k + a.eps);
    for (int64_t c = lx; c < a.chunks; c += tpr) {
      Chunk<T> xv, rv;
      const int n = chunk_len(c, a.k);
      load_chunk(xv, x, c, n);
      if (r) load_chunk(rv, r, c, n);
      else rv.zero();
      finish(xv, rv, c, n, rstd);
    }
  }
}

int log2_up(int64_t v, int lo, int hi) {
  int b = lo;
  while (b < hi && (int64_t(1) << b) < v) ++b;
  return b;
}

// Workgroups a launch holds at most (a grid's threads are counted in 32 bits):
// taller matrices take several launches over slabs of rows.
constexpr int64_t kMaxBlocks = int64_t(1) << 21;

// Rows of at least 4 chunks; segments of up to 256 x UNR chunks.  Calls
// launch(first row, rows, workgroups) for each slab.
template <typename F>
hipError_t over_slabs(int64_t M, int64_t k, int unr, RowGrid *g, F &&launch) {
  g->chunks = (k + kBlock - 1) / kBlock * 4;
  g->log_tx = log2_up((g->chunks + unr - 1) / unr, 2, 8);
  const int64_t per = (int64_t)unr << g->log_tx;
  g->nseg = (uint32_t)((g->chunks + per - 1) / per);
  const int64_t rows = kThreads >> g->log_tx;
  const int64_t slab = rows * std::max<int64_t>(1, kMaxBlocks / g->nseg);
  for (int64_t m0 = 0; m0 < M; m0 += slab) {
    const int64_t n = std::min(slab, M - m0);
    launch(m0, n, (unsigned)((n + rows - 1) / rows * g->nseg));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int FMT>
hipError_t quantize_t(const MxQuantArgs &a, hipStream_t st) {
  constexpr int UNR = 4;
  RowGrid g;
  return over_slabs(a.M, a.k, UNR, &g, [&](int64_t m0, int64_t n, unsigned blocks) {
    hipLaunchKernelGGL((k_mx_quantize<T, FMT, UNR>), dim3(blocks), dim3(kThreads), 0, st,
                       (const T *)a.x + m0 * a.ldx, a.ldx, n, a.k, g, a.q + m0 * a.ldq, a.ldq,
                       a.sc + m0 * a.lds, a.lds);
  });
}

template <typename T, int FMT>
hipError_t dequantize_t(const MxQuantArgs &a, hipStream_t st) {
  constexpr int UNR = 4;
  RowGrid g;
  return over_slabs(a.M, a.k, UNR, &g, [&](int64_t m0, int64_t n, unsigned blocks) {
    hipLaunchKernelGGL((k_mx_dequantize<T, FMT, UNR>), dim3(blocks), dim3(kThreads), 0, st,
                       a.q + m0 * a.ldq, a.ldq, a.sc + m0 * a.lds, a.lds, n, a.k, g,
                       (T *)const_cast<void *>(a.x) + m0 * a.ldx, a.ldx);
  });
}

template <typename T, int FMT>
hipError_t rmsnorm_t(NormArgs a, hipStream_t st) {
  constexpr int CMAX = 4;
  // threads per row: up to four chunks each; rows past 1024 x 4 chunks are
  // read twice
  a.log_tpr = log2_up((a.chunks + CMAX - 1) / CMAX, 2, 10);
  const int64_t per = (a.chunks + (int64_t(1) << a.log_tpr) - 1) >> a.log_tpr;
  // several rows to a workgroup while a row takes at most a wave
  const int block = a.log_tpr > 6 ? 1 << a.log_tpr : kThreads;
  const int64_t rows = block >> a.log_tpr;
  const int64_t M = a.M;
  const NormArgs all = a;
  for (int64_t m0 = 0; m0 < M; m0 += rows * kMaxBlocks) {
    a.M = std::min(rows * kMaxBlocks, M - m0);
    a.x = (const T *)all.x + m0 * a.ldx;
    if (all.res) a.res = (const T *)all.res + m0 * a.ldr;
    if (all.h) a.h = (T *)all.h + m0 * a.ldh;
    if (all.y) a.y = (T *)all.y + m0 * a.ldy;
    if (FMT) {
      a.q = all.q + m0 * a.ldq;
      a.sc = all.sc + m0 * a.lds;
    }
    const dim3 grid((unsigned)((a.M + rows - 1) / rows)), blk(block);
    if (per <= 1) hipLaunchKernelGGL((k_rmsnorm<T, FMT, 1>), grid, blk, 0, st, a);
    else if (per <= 2) hipLaunchKernelGGL((k_rmsnorm<T, FMT, 2>), grid, blk, 0, st, a);
    else if (per <= CMAX) hipLaunchKernelGGL((k_rmsnorm<T, FMT, CMAX>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_rmsnorm<T, FMT, 0>), grid, blk, 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs &a, hipStream_t st) {
  if (a.M <= 0) return hipSuccess;
  if (a.dtype == LORA_DTYPE_BF16)
    return a.fmt == kFp8 ? quantize_t<uint16_t, kFp8>(a, st) : quantize_t<uint16_t, kFp4>(a, st);
  return a.fmt == kFp8 ? quantize_t<float, kFp8>(a, st) : quantize_t<float, kFp4>(a, st);
}

hipError_t launch_mx_dequantize(const MxQuantArgs &a, hipStream_t st) {
  if (a.M <= 0) return hipSuccess;
  if (a.dtype == LORA_DTYPE_BF16)
    return a.fmt == kFp8 ? dequantize_t<uint16_t, kFp8>(a, st) : dequantize_t<uint16_t, kFp4>(a, st);
  return a.fmt == kFp8 ? dequantize_t<float, kFp8>(a, st) : dequantize_t<float, kFp4>(a, st);
}

hipError_t launch_rmsnorm(const RmsNormArgs &n, hipStream_t st) {
  if (n.M <= 0) return hipSuccess;
  NormArgs a{};
  a.x = n.x; a.res = n.res; a.w = n.w; a.h = n.h; a.y = n.y;
  a.q = n.q; a.sc = n.sc;
  a.ldx = n.ldx; a.ldr = n.ldr; a.ldh = n.ldh; a.ldy = n.ldy; a.ldq = n.ldq; a.lds = n.lds;
  a.M = n.M; a.k = n.k;
  a.chunks = (n.k + kBlock - 1) / kBlock * 4;
  a.eps = (double)n.eps;
  a.inv_k = 1.0 / (double)n.k;
  if (n.dtype == LORA_DTYPE_BF16) {
    if (n.fmt == kFp8) return rmsnorm_t<uint16_t, kFp8>(a, st);
    if (n.fmt == kFp4) return rmsnorm_t<uint16_t, kFp4>(a, st);
    return rmsnorm_t<uint16_t, 0>(a, st);
  }
  if (n.fmt == kFp8) return rmsnorm_t<float, kFp8>(a, st);
  if (n.fmt == kFp4) return rmsnorm_t<float, kFp4>(a, st);
  return rmsnorm_t<float, 0>(a, st);
}

}  // namespace lora
