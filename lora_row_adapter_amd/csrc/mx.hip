// mx.hip -- microscaled quantising and reading back, and the root-mean-square
// norm with a microscaled output (include/lora_mx.h).
//
// All three are one pass over the data and bound by its bytes.  A row is cut
// into chunks of 16 bytes, one lane each, so a block of 32 elements is four
// (bf16) or eight (fp32) lanes: its largest magnitude takes two or three DPP
// moves, and a wave's loads and stores of values are contiguous.
#include <algorithm>

#include "mx_device.hpp"
#include "plan_body.hpp"

namespace lora {

using namespace mx;

namespace {

constexpr int kThreads = 256;

// A workgroup covers (its threads >> log_tx) rows x 1 << log_tx chunk columns
// in each of UNR steps along the row; workgroups run over column segments
// first.
struct RowGrid {
  int32_t log_tx;
  uint32_t nseg;   // column segments per row group
  int64_t chunks;  // chunks per row, whole blocks
};

struct Rows {  // a dense matrix and its microscaled form
  void *x;
  int64_t ldx;
  uint8_t *q, *sc;
  int64_t ldq, lds;
  int64_t M, k;
};

template <typename T, int FMT, int UNR, int NT>
__device__ __forceinline__ void quantize_rows(const Rows &a, const RowGrid &g, uint32_t block) {
  using C = Chunk<T>;
  const int lx = threadIdx.x & ((1 << g.log_tx) - 1);
  const uint32_t grp = block / g.nseg, seg = block - grp * g.nseg;
  const int64_t m = (int64_t)grp * (NT >> g.log_tx) + (threadIdx.x >> g.log_tx);
  if (m >= a.M) return;  // whole blocks leave: a row has at least a block's lanes
  const int64_t c0 = (int64_t)seg * (UNR << g.log_tx) + lx;
  const T *row = (const T *)a.x + m * a.ldx;
  C v[UNR];
#pragma unroll
  for (int i = 0; i < UNR; ++i) {
    const int64_t c = c0 + ((int64_t)i << g.log_tx);
    v[i].load(row, c, C::len(c, a.k));
  }
#pragma unroll
  for (int i = 0; i < UNR; ++i) {
    const int64_t c = c0 + ((int64_t)i << g.log_tx);
    float f[C::kElems];
#pragma unroll
    for (int e = 0; e < C::kElems; ++e) f[e] = v[i].get(e);
    quantise_chunk<FMT>(f, c, c < g.chunks, a.q + m * a.ldq, a.sc + m * a.lds);
  }
}

// 9216 x 8192 fp32 to fp4 59 us (5.8 TB/s), 8192 x 4096 bf16 to fp8 18.7 us
// (5.4 TB/s), 1 x 8192 2 us.  UNR loads a thread are in flight before the
// first is used: with one, 69 and 21.5 us.
template <typename T, int FMT, int UNR>
__global__ __launch_bounds__(kThreads) void k_mx_quantize(Rows a, RowGrid g) {
  quantize_rows<T, FMT, UNR, kThreads>(a, g, blockIdx.x);
}

// The codes' values are exact in fp32, and so is their product with the scale
// (but past fp32's range): one rounding, to bf16 where that is asked for.
// 9216 x 8192 fp32 from fp4 48 us (7 TB/s), 8192 x 4096 bf16 from fp8 15.8
// us (6.4 TB/s), 1 x 8192 2 us.
template <typename T, int FMT, int UNR>
__global__ __launch_bounds__(kThreads) void k_mx_dequantize(Rows a, RowGrid g) {
  using C = Chunk<T>;
  constexpr int N = C::kElems;
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const int lx = threadIdx.x & ((1 << g.log_tx) - 1);
  const uint32_t grp = blockIdx.x / g.nseg, seg = blockIdx.x - grp * g.nseg;
  const int64_t m = (int64_t)grp * (kThreads >> g.log_tx) + (threadIdx.x >> g.log_tx);
  if (m >= a.M) return;
  const int64_t c0 = (int64_t)seg * (UNR << g.log_tx) + lx;
  const uint8_t *qrow = a.q + m * a.ldq, *srow = a.sc + m * a.lds;
  uint32_t w[UNR][2], s[UNR];  // N codes of fp8 or fp4
#pragma unroll
  for (int i = 0; i < UNR; ++i) {
    const int64_t c = c0 + ((int64_t)i << g.log_tx);
    w[i][0] = w[i][1] = s[i] = 0;
    if (c < g.chunks) {
      if constexpr (FMT == kFp8) __builtin_memcpy(w[i], __builtin_assume_aligned(qrow + c * N, N), N);
      else __builtin_memcpy(w[i], __builtin_assume_aligned(qrow + c * (N / 2), N / 2), N / 2);
      s[i] = srow[c / C::kLanes];
    }
  }
#pragma unroll
  for (int i = 0; i < UNR; ++i) {
    const int64_t c = c0 + ((int64_t)i << g.log_tx);
    const float f = scale_value(s[i]);
    C o;
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      f32x2_t lo, hi;
      if constexpr (FMT == kFp8) {
        lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i][e / 4], false);
        hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i][e / 4], true);
      } else if (e == 0) {
        lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i][0], 1.0f, 0);
        hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i][0], 1.0f, 1);
      } else {
        lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i][0], 1.0f, 2);
        hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i][0], 1.0f, 3);
      }
      o.set2(e, lo[0] * f, lo[1] * f);
      o.set2(e + 2, hi[0] * f, hi[1] * f);
    }
    o.store((T *)a.x + m * a.ldx, c, C::len(c, a.k));
  }
}

// v rounded to fp32 "to odd": toward zero, with the last bit set when that
// was inexact.  A further rounding of the result to fewer bits than fp32
// minus two is then the correct rounding of v itself.  What rounds to nearest
// as an infinity is one (and its block's scale NaN, as its value in fp32).
__device__ __forceinline__ float to_odd(double v) {
  const float f = (float)v;
  const double d = (double)f;
  uint32_t b = __float_as_uint(f);
  if (d != v && !(b & 1u) && fabsf(f) < __builtin_inff()) b += fabs(d) > fabs(v) ? 0xffffffffu : 1u;
  return __uint_as_float(b);
}

struct NormArgs {
  const void *x, *res, *w;
  void *h, *y;
  uint8_t *q, *sc;
  int64_t ldx, ldr, ldh, ldy, ldq, lds;
  int64_t M, k, chunks;
  double eps, inv_k;
  int32_t log_tpr;  // threads per row (a power of two, at most the workgroup's)
};

// Sum over the threads of a row, which are 1 << log_tpr neighbours; rows of
// several waves put their waves' sums in `red`.
__device__ __forceinline__ double row_sum(double s, int log_tpr, double *red) {
  const int in_wave = log_tpr < 6 ? log_tpr : 6;
  for (int i = 0; i < in_wave; ++i) s += __shfl_xor(s, 1 << i, 64);
  if (log_tpr > 6) {
    const int nw = 1 << (log_tpr - 6), wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = s;
    __syncthreads();
    s = 0;
    for (int i = 0; i < nw; ++i) s += red[(wave & ~(nw - 1)) + i];
  }
  return s;
}

// The rows of workgroup `block`, one per 1 << log_tpr threads:
//   h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.
// The squares are summed in 64 bits (a conversion and an addition per input
// cost about what the memory takes anyway).  The outputs are those of one
// rounding of the 64-bit y, but computing them in 64 bits throughout costs
// 143 us, not 113, at 8192 x 8192 bf16 with a residual (604 MB, 5.3 TB/s):
// they are computed in fp32 and redone in 64 bits where the two could differ.
// NC > 0: each thread keeps its NC chunks of x and the residual in registers,
// so every input is read once; NC == 0: rows too long for that are read twice.
template <typename T, int FMT, int NC, bool RES>
__device__ __forceinline__ void rmsnorm_rows(const NormArgs &a, uint32_t block, double *red) {
  using C = Chunk<T>;
  constexpr int N = C::kElems;
  const int tpr = 1 << a.log_tpr;
  const int lx = threadIdx.x & (tpr - 1);
  const int64_t at = (int64_t)block * (blockDim.x >> a.log_tpr) + (threadIdx.x >> a.log_tpr);
  // rows past the last redo it and write nothing: every thread meets the barrier
  const bool live = at < a.M;
  const int64_t m = live ? at : a.M - 1;
  const T *x = (const T *)a.x + m * a.ldx;
  const T *r = RES ? (const T *)a.res + m * a.ldr : nullptr;
  const T *w = (const T *)a.w;
  T *h = a.h ? (T *)a.h + m * a.ldh : nullptr;
  T *y = a.y ? (T *)a.y + m * a.ldy : nullptr;

  auto load = [&](int64_t c, int n, C &xv, C &rv) {
    xv.load(x, c, n);
    if constexpr (RES) rv.load(r, c, n);
  };
  auto squares = [&](const C &xv, const C &rv, double s) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      double v = (double)xv.get(e);
      if constexpr (RES) v += (double)rv.get(e);
      s = fma(v, v, s);
    }
    return s;
  };
  auto finish = [&](const C &xv, const C &rv, const C &wv, int64_t c, int n, double rstd) {
    C o;
    float hs[N], f[N];
    // for bf16 rounded twice, to 24 and to 8 bits, but as if once: 24 >= 2 * 8 + 2
#pragma unroll
    for (int e = 0; e < N; ++e) hs[e] = RES ? xv.get(e) + rv.get(e) : xv.get(e);
    if (h != nullptr) {
#pragma unroll
      for (int e = 0; e < N; e += 2) o.set2(e, hs[e], hs[e + 1]);
      o.store(h, c, n);
    }
    auto exact = [&](int e) {
      double v = (double)xv.get(e);
      if constexpr (RES) v += (double)rv.get(e);
      return v * rstd * (double)wv.get(e);
    };
    // `near` is small where a value's low 15 bits are within `kOff` of 0, that
    // is near a value that bf16 or a code represents or a midpoint of two;
    // below 2^-100 midpoints lie elsewhere
    uint32_t near = ~0u;
    float low = __builtin_inff();
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        f[e] = (float)exact(e);
        near = min(near, __float_as_uint(f[e]) << 17);
        low = fminf(low, fabsf(f[e]));
      }
      if (y != nullptr) {
#pragma unroll
        for (int e = 0; e < N; e += 2) o.set2(e, f[e], f[e + 1]);
        o.store(y, c, n);
      }
      if (FMT && (near == 0 || !(low >= 0x1p-100f))) {
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = to_odd(exact(e));
      }
    } else {
      constexpr uint32_t kOff = 5;  // four roundings of half a step each, relative: four steps at most
      const float rs = rstd > 0x1p-100 && rstd < 0x1p100 ? (float)rstd : __builtin_nanf("");
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float v = hs[e] * rs;
        f[e] = v * wv.get(e);
        near = min(near, (__float_as_uint(f[e]) + kOff) << 17);
        low = fminf(low, fminf(fabsf(v), fabsf(f[e])));
      }
      if (near < (2 * kOff + 1) << 17 || !(low >= 0x1p-100f)) {
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = to_odd(exact(e));
      }
      if (y != nullptr) {
#pragma unroll
        for (int e = 0; e < N; e += 2) o.set2(e, f[e], f[e + 1]);
        o.store(y, c, n);
      }
    }
    if constexpr (FMT != 0) {
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = e < n ? f[e] : 0.f;  // 0 * inf past the row's end
      quantise_chunk<FMT>(f, c, true, a.q + m * a.ldq, a.sc + m * a.lds);
    }
  };

  double s = 0;
  if constexpr (NC > 0) {
    C xv[NC], rv[NC], wv[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t c = ((int64_t)i << a.log_tpr) + lx;
      load(c, C::len(c, a.k), xv[i], rv[i]);
    }
    // the weight too, ahead of the sum: one row's time is its loads' latency
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t c = ((int64_t)i << a.log_tpr) + lx;
      wv[i].load(w, c, C::len(c, a.k));
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) s = squares(xv[i], rv[i], s);
    s = row_sum(s, a.log_tpr, red);
    if (!live) return;
    const double rstd = 1.0 / sqrt(s * a.inv_k + a.eps);
    // past 16 elements a thread none of the sum's 64-bit values stay for the
    // outputs: 110 registers, not 128 and 80 spilled (8192 x 8192 bf16 by 256
    // threads a row: 127 us, not 322); up to 16 they do (112 us, not 124)
    if constexpr (NC * N > 16) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        xv[i].hide();
        if constexpr (RES) rv[i].hide();
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t c = ((int64_t)i << a.log_tpr) + lx;
      if (c < a.chunks) finish(xv[i], rv[i], wv[i], c, C::len(c, a.k), rstd);
    }
  } else {
    C xv, rv;
    for (int64_t c = lx; c < a.chunks; c += tpr) {
      load(c, C::len(c, a.k), xv, rv);
      s = squares(xv, rv, s);
    }
    s = row_sum(s, a.log_tpr, red);
    if (!live) return;
    const double rstd = 1.0 / sqrt(s * a.inv_k + a.eps);
    for (int64_t c = lx; c < a.chunks; c += tpr) {
      const int n = C::len(c, a.k);
      load(c, n, xv, rv);
      C wv;
      wv.load(w, c, n);
      finish(xv, rv, wv, c, n, rstd);
    }
  }
}

template <typename T, int FMT, int NC, bool RES>
__global__ __launch_bounds__(1024) void k_rmsnorm(NormArgs a) {
  __shared__ double red[16];
  rmsnorm_rows<T, FMT, NC, RES>(a, blockIdx.x, red);
}

// The layer's plan beside the rows' work: workgroup 0 runs it, the others the
// rows.  It needs the ids alone, so it hides behind the norm (or the
// quantising) without a stream of its own, whose fork and join cost 6 us:
// a layer of 512 rows, 8192 -> 9216, goes from 95 to 87 us, one of 8192 rows,
// 4096 -> 4096, from 158 to 151.
template <int FMT, int NT, bool RES>
__global__ __launch_bounds__(NT) void k_rmsnorm_plan(NormArgs a, PlanArgs plan, uint32_t lds_bytes) {
  extern __shared__ __attribute__((aligned(16))) uint8_t plan_lds[];
  __shared__ double red[16];
  if (blockIdx.x == 0) plan_detail::plan_body<NT>(plan, plan_lds, lds_bytes);
  else rmsnorm_rows<uint16_t, FMT, 2, RES>(a, blockIdx.x - 1, red);
}
template <int FMT, int NT>
__global__ __launch_bounds__(NT) void k_mx_quantize_plan(Rows a, RowGrid g, PlanArgs plan, uint32_t lds_bytes) {
  extern __shared__ __attribute__((aligned(16))) uint8_t plan_lds[];
  if (blockIdx.x == 0) plan_detail::plan_body<NT>(plan, plan_lds, lds_bytes);
  else quantize_rows<uint16_t, FMT, 4, NT>(a, g, blockIdx.x - 1);
}

int log2_up(int64_t v, int lo, int hi) {
  int b = lo;
  while (b < hi && (int64_t(1) << b) < v) ++b;
  return b;
}

// Workgroups a launch holds at most (a grid's threads are counted in 32 bits):
// taller matrices take several launches over slabs of rows.
constexpr int64_t kMaxBlocks = int64_t(1) << 21;

// Grid of k_mx_quantize / k_mx_dequantize, UNR steps a thread.
template <typename T>
RowGrid row_grid(int64_t k, int unr) {
  RowGrid g;
  constexpr int lanes = Chunk<T>::kLanes;
  g.chunks = (k + kBlock - 1) / kBlock * lanes;
  g.log_tx = log2_up((g.chunks + unr - 1) / unr, lanes == 4 ? 2 : 3, 8);
  const int64_t per = (int64_t)unr << g.log_tx;
  g.nseg = (uint32_t)((g.chunks + per - 1) / per);
  return g;
}

Rows rows_of(const MxQuantArgs &a) {
  return Rows{const_cast<void *>(a.x), a.ldx, a.q, a.sc, a.ldq, a.lds, a.M, a.k};
}

// launch(rows, workgroups) for each slab of rows.
template <typename T, typename F>
hipError_t over_slabs(const MxQuantArgs &a, const RowGrid &g, F &&launch) {
  const int64_t rows = kThreads >> g.log_tx;
  const int64_t slab = rows * std::max<int64_t>(1, kMaxBlocks / g.nseg);
  for (int64_t m0 = 0; m0 < a.M; m0 += slab) {
    Rows r = rows_of(a);
    r.M = std::min(slab, a.M - m0);
    r.x = (T *)r.x + m0 * r.ldx;
    r.q += m0 * r.ldq;
    r.sc += m0 * r.lds;
    launch(r, (unsigned)((r.M + rows - 1) / rows * g.nseg));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int FMT>
hipError_t quantize_t(const MxQuantArgs &a, hipStream_t st) {
  constexpr int UNR = sizeof(T) == 4 ? 2 : 4;  // 9216 x 8192 fp32: 60 us, with 4 63, 1 69
  const RowGrid g = row_grid<T>(a.k, UNR);
  return over_slabs<T>(a, g, [&](const Rows &r, unsigned blocks) {
    hipLaunchKernelGGL((k_mx_quantize<T, FMT, UNR>), dim3(blocks), dim3(kThreads), 0, st, r, g);
  });
}

template <typename T, int FMT>
hipError_t dequantize_t(const MxQuantArgs &a, hipStream_t st) {
  constexpr int UNR = 4;
  const RowGrid g = row_grid<T>(a.k, UNR);
  return over_slabs<T>(a, g, [&](const Rows &r, unsigned blocks) {
    hipLaunchKernelGGL((k_mx_dequantize<T, FMT, UNR>), dim3(blocks), dim3(kThreads), 0, st, r, g);
  });
}

// Threads per row and chunks per thread (0: the row is read twice).  16
// elements a thread keep most loads in flight for a workgroup that waits
// once: 8192 x 8192 bf16 with a residual and fp8 codes takes 112 us, with 8
// elements 165, 32 127; 512 rows 8.9, 11.4 and 10.4 us; 1000 x 5003 fp32
// without a residual, fp4 codes 13.5 us, with 8 elements 18.
struct NormShape {
  int log_tpr, nc, block;
};
template <typename T>
NormShape norm_shape(int64_t chunks) {
  NormShape s;
  constexpr int nc = 16 / Chunk<T>::kElems;
  s.log_tpr = log2_up((chunks + nc - 1) / nc, Chunk<T>::kLanes == 4 ? 2 : 3, 10);
  const int64_t per = (chunks + (int64_t(1) << s.log_tpr) - 1) >> s.log_tpr;
  s.nc = per <= 2 ? 2 : per <= 4 ? 4 : 0;
  s.block = std::max(kThreads, 1 << s.log_tpr);
  return s;
}

template <typename T, int FMT>
hipError_t rmsnorm_t(NormArgs a, hipStream_t st) {
  const NormShape sh = norm_shape<T>(a.chunks);
  a.log_tpr = sh.log_tpr;
  const int64_t rows = sh.block >> sh.log_tpr;
  const NormArgs all = a;
  for (int64_t m0 = 0; m0 < all.M; m0 += rows * kMaxBlocks) {
    a.M = std::min(rows * kMaxBlocks, all.M - m0);
    a.x = (const T *)all.x + m0 * a.ldx;
    if (all.res) a.res = (const T *)all.res + m0 * a.ldr;
    if (all.h) a.h = (T *)all.h + m0 * a.ldh;
    if (all.y) a.y = (T *)all.y + m0 * a.ldy;
    if (FMT) {
      a.q = all.q + m0 * a.ldq;
      a.sc = all.sc + m0 * a.lds;
    }
    const dim3 grid((unsigned)((a.M + rows - 1) / rows)), blk(sh.block);
    const auto kernel = sh.nc == 2   ? (a.res ? k_rmsnorm<T, FMT, 2, true> : k_rmsnorm<T, FMT, 2, false>)
                        : sh.nc == 4 ? (a.res ? k_rmsnorm<T, FMT, 4, true> : k_rmsnorm<T, FMT, 4, false>)
                                     : (a.res ? k_rmsnorm<T, FMT, 0, true> : k_rmsnorm<T, FMT, 0, false>);
    hipLaunchKernelGGL(kernel, grid, blk, 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The plan beside the rows' work is the one for few adapters, whose LDS (2 to
// 10 KiB up to 1024 rows, 48 KiB for 8192) every workgroup of the launch is
// given: past 1024 rows the workgroups are of 1024 threads, of which a CU
// holds two at most anyway, and the plan is as fast as its own kernel.
constexpr int kPlanAdapters = 64;
constexpr int64_t kPlanCols = int64_t(1) << 20;  // one launch, so a grid within 32 bits of threads

template <int FMT, int NT>
void norm_plan(const NormArgs &a, const PlanArgs &p, hipStream_t st) {
  const size_t lds = plan_detail::plan_small_lds(p.M, NT);
  const int64_t rows = NT >> a.log_tpr;
  hipLaunchKernelGGL((a.res ? k_rmsnorm_plan<FMT, NT, true> : k_rmsnorm_plan<FMT, NT, false>), dim3((unsigned)((a.M + rows - 1) / rows + 1)), dim3(NT),
                     lds, st, a, p, (uint32_t)lds);
}
template <int FMT>
void norm_plan(const NormArgs &a, int block, const PlanArgs &p, hipStream_t st) {
  if (p.M > 1024 || block > 512) norm_plan<FMT, 1024>(a, p, st);
  else if (block > 256) norm_plan<FMT, 512>(a, p, st);
  else norm_plan<FMT, 256>(a, p, st);
}

template <int FMT, int NT>
void quantize_plan(const MxQuantArgs &a, const PlanArgs &p, hipStream_t st) {
  const RowGrid g = row_grid<uint16_t>(a.k, 4);
  const size_t lds = plan_detail::plan_small_lds(p.M, NT);
  const int64_t rows = NT >> g.log_tx;
  hipLaunchKernelGGL((k_mx_quantize_plan<FMT, NT>), dim3((unsigned)((a.M + rows - 1) / rows * g.nseg + 1)),
                     dim3(NT), lds, st, rows_of(a), g, p, (uint32_t)lds);
}
template <int FMT>
void quantize_plan(const MxQuantArgs &a, const PlanArgs &p, hipStream_t st) {
  if (p.M > 1024) quantize_plan<FMT, 1024>(a, p, st);
  else quantize_plan<FMT, kThreads>(a, p, st);
}
}  // namespace

bool mx_runs_plan(int64_t M, int64_t k, int32_t n_adapters, bool norm) {
  if (M < 1 || M > kPlanMaxRows || k > kPlanCols || n_adapters > kPlanAdapters) return false;
  return !norm || norm_shape<uint16_t>((k + kBlock - 1) / kBlock * 4).nc == 2;
}

hipError_t launch_mx_quantize(const MxQuantArgs &a, hipStream_t st, const PlanArgs *plan) {
  if (a.M <= 0) return hipSuccess;
  if (plan != nullptr) {
    if (a.dtype != LORA_DTYPE_BF16 || !mx_runs_plan(a.M, a.k, plan->S, false)) return hipErrorInvalidValue;
    if (a.fmt == kFp8) quantize_plan<kFp8>(a, *plan, st);
    else quantize_plan<kFp4>(a, *plan, st);
    return hipGetLastError();
  }
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

hipError_t launch_rmsnorm(const RmsNormArgs &n, hipStream_t st, const PlanArgs *plan) {
  if (n.M <= 0) return hipSuccess;
  NormArgs a{};
  a.x = n.x; a.res = n.res; a.w = n.w; a.h = n.h; a.y = n.y;
  a.q = n.q; a.sc = n.sc;
  a.ldx = n.ldx; a.ldr = n.ldr; a.ldh = n.ldh; a.ldy = n.ldy; a.ldq = n.ldq; a.lds = n.lds;
  a.M = n.M; a.k = n.k;
  a.chunks = (n.k + kBlock - 1) / kBlock * (n.dtype == LORA_DTYPE_BF16 ? 4 : 8);
  a.eps = (double)n.eps;
  a.inv_k = 1.0 / (double)n.k;
  if (plan != nullptr) {
    if (n.dtype != LORA_DTYPE_BF16 || n.fmt == 0 || !mx_runs_plan(n.M, n.k, plan->S, true))
      return hipErrorInvalidValue;
    const NormShape s = norm_shape<uint16_t>(a.chunks);
    a.log_tpr = s.log_tpr;
    if (n.fmt == kFp8) norm_plan<kFp8>(a, s.block, *plan, st);
    else norm_plan<kFp4>(a, s.block, *plan, st);
    return hipGetLastError();
  }
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
