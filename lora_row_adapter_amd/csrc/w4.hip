// w4.hip -- the 4-bit base weight of include/lora_w4.h: laying it out, reading
// it back, and the product
//   y[m, n] = sum_g s[n, g] (sum_{j in g} x[m, j] q[n, j] - z[n, g] sum_{j in g} x[m, j])
//
// A code in a byte is an E4M3 number, q 2^-9 exactly (subnormals and the first
// binade lie on one line), so gfx950's scaled conversion turns two codes into
// two bf16 in one instruction at the full rate: seven instructions for eight
// codes.  The matrix instruction multiplies them with x as they are, and x
// with a column of ones for the group's sum X of x; then
//   tot += s (acc - z X)
// in fp32: no weight is rounded.
#include <algorithm>
#include <type_traits>

#include "plan_body.hpp"

namespace lora {

namespace {

__device__ __forceinline__ float scale_of(uint32_t w) { return __uint_as_float(w & ~31u); }

// The codes of one dword as the matrix instruction's eight bf16: columns 0 - 3
// from the low nibbles of its bytes, 4 - 7 from the high ones.
__device__ __forceinline__ bf16x8_t codes(uint32_t w) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------- layout
// One workgroup a record: 256 threads a dword of codes each, then its scales.  Done
// once for a weight, so codes are read byte by byte, as any alignment of theirs
// allows: 9216 x 8192 70 us, 1.1 TB/s.
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
    for (int p = 0; p < 4; ++p) {  // columns 2p and 2p + 1
      const int64_t j = j0 + 2 * p;
      if (j < a.k) {
        const uint32_t b = row[j >> 1];
        const int at = 16 * (p & 1) + 4 * (p >> 1);
        w |= (b & 15u) << at | (b >> 4) << (at + 8);
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

// A workgroup reads kDqRecords records of 16 rows back; of each, a thread takes
// a dword of codes (eight columns of a row) and sixteen threads a row's 128
// columns.  All of a thread's loads go ahead of its stores.  Bound by its bytes:
// 9216 x 8192 to bf16 37 - 45 us, 4.2 TB/s and more (a part stays in the last-level
// cache), to fp32 102 us, 3.4 TB/s (a thread's 32 bytes are two stores).
constexpr int kDqRecords = 8;
template <typename T>
__global__ __launch_bounds__(256) void k_w4_dequantize(W4Args a, int32_t per_row) {
  const int64_t tile = blockIdx.x / per_row;
  const int blk0 = (int)(blockIdx.x - tile * per_row) * kDqRecords;
  const uint8_t *in = a.w + (tile * a.nb + blk0) * w4_record(a.sg);
  const int t = threadIdx.x, row = t >> 4, i = (t >> 2) & 3, h = t & 3;
  const int64_t n = tile * 16 + row;
  if (n >= a.d) return;
  const int at = ((h * 16 + row) * 4 + i) * 4, sat = (int)kW4Codes + ((i * a.sg >> 2) * 16 + row) * 4;
  uint32_t w[kDqRecords], sw[kDqRecords];
#pragma unroll
  for (int r = 0; r < kDqRecords; ++r) {
    const uint8_t *rec = in + min(r, a.nb - 1 - blk0) * w4_record(a.sg);
    w[r] = *reinterpret_cast<const uint32_t *>(rec + at);
    sw[r] = *reinterpret_cast<const uint32_t *>(rec + sat);
  }
#pragma unroll
  for (int r = 0; r < kDqRecords; ++r) {
    const int64_t j0 = (int64_t)(blk0 + r) * 128 + 32 * i + 8 * h;
    if (j0 >= a.k) return;
    const float s = scale_of(sw[r]);
    const int z = (int)(sw[r] & 31u);
    // 19 bits by 5: the products are exact
    T o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = s * (float)((int)((w[r] >> (8 * (e & 3) + (e & 4))) & 15u) - z);
      if constexpr (sizeof(T) == 2) o[e] = f32_to_bf16_bits(v);
      else o[e] = v;
    }
    T *y = (T *)a.y + n * a.ldy + j0;
    const int left = (int)min((int64_t)8, a.k - j0);
    if (left == 8 && ((uintptr_t)y & 15) == 0) {
#pragma unroll
      for (int c = 0; c < (int)sizeof(T) / 2; ++c)
        reinterpret_cast<uint4 *>(y)[c] = reinterpret_cast<const uint4 *>(o)[c];
    } else {
      for (int e = 0; e < left; ++e) y[e] = o[e];
    }
  }
}

// ---------------------------------------------------------------- few rows
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
// Past every buffer: loads give zeros.  Either offset may be it: the two are added
// without wrapping (read back on the machine, from a buffer that goes on).
constexpr uint32_t kOob = 0xFFFFFFF0u;

__device__ __forceinline__ bf16x8_t ones8() {
  return __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, 0x00020000);
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}
// The fragments of FM 16-row tiles for two steps of 32 columns, at a0 and a1
// and 2 KiB on for each tile, and the wait for them: one statement, as the
// compiler would wait for every load into LDS ahead of a read of its own.
template <int FM>
__device__ __forceinline__ void read_half(uint32_t a0, uint32_t a1, u32x4_t (&x)[2][FM]) {
  static_assert(FM == 1 || FM == 2 || FM == 4, "tiles");
  if constexpr (FM == 1)
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(x[0][0]), "=&v"(x[1][0]) : "v"(a0), "v"(a1) : "memory");
  else if constexpr (FM == 2)
    asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:2048\n\t"
                 "ds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[1][0]), "=&v"(x[1][1]) : "v"(a0), "v"(a1) : "memory");
  else
    asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:2048\n\tds_read_b128 %2, %8 offset:4096\n\t"
                 "ds_read_b128 %3, %8 offset:6144\n\tds_read_b128 %4, %9\n\tds_read_b128 %5, %9 offset:2048\n\t"
                 "ds_read_b128 %6, %9 offset:4096\n\tds_read_b128 %7, %9 offset:6144\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[0][2]), "=&v"(x[0][3]), "=&v"(x[1][0]), "=&v"(x[1][1]),
                   "=&v"(x[1][2]), "=&v"(x[1][3]) : "v"(a0), "v"(a1) : "memory");
}

// kWith: kPlan: workgroup 0 runs the layer's plan; kLora: the adapters' part is
// added (see LoraPart), and workgroup 0 runs the plan where it is to be made.
enum With { kNone, kPlan, kLora };
struct Nothing {};
struct LoraWith {
  W4Lora lora;
  PlanArgs plan;
  int32_t planned;
};
template <With kWith>
using with_t = std::conditional_t<kWith == kPlan, PlanArgs, std::conditional_t<kWith == kLora, LoraWith, Nothing>>;

// The adapters' part of a workgroup's rows and columns, t B_s^T, is the work of
// lora_waves more waves: what it waits for, one after the other (the rows'
// adapters, then their B), passes while the others stream W.  8192 x 9216, one row: 9
// us without it, 10 so, 13 - 14 where the same waves did it before, in or after their
// own records; 16 rows of 12 adapters: 14 so, 16 - 19.  For 33 to 64 rows, in two tiles,
// it took as long as the product, a plan and two kernels more, or up to 1.3 of it.
template <int FM, int FN>
constexpr int lora_waves = FM * FN <= 3 ? 8 : 4;  // as many as the sums of W's waves leave registers for

// Each distinct adapter and 16 columns are one unit, kAhead of them with their B on its
// way at once.  A product is taken for all rows of a tile and added to those of that
// adapter alone, so no adapter's values reach another's rows.
template <int FM, int FN>
struct LoraPart {
  static constexpr int ROWS = 16 * FM, kAhead = 3;
  const W4Lora &l;
  const int m0, n0, lane, r, h;
  const int M, Rp;
  int own, lrank;            // of row m0 + lane
  int q, k0;                 // the slice, the first of 64 ranks
  int first, d;              // this lane's first column in the slice, its columns
  uint64_t of[kAhead];       // units: rows, 16 columns, adapter, rank, B
  int at[kAhead], us[kAhead], ur[kAhead];
  u32x4_t b[kAhead][2];
  u32x4_t t[2][FM][2];       // high and low parts

  __device__ __forceinline__ LoraPart(const W4Lora &l, int m0, int n0)
      : l(l), m0(m0), n0(n0), lane(threadIdx.x & 63), r(lane & 15), h(lane >> 4), M(l.M), Rp(l.Rp) {}

  // A value of each row: 0: its adapter, 1 + q: its rank in slice q.
  __device__ __forceinline__ int of_row(const int32_t *rows, int i) const {
    return rows[i * M + m0 + min(lane, min(ROWS, M - m0) - 1)];
  }
  __device__ __forceinline__ void load_t() {
    const uint32_t bytes = (uint32_t)(l.n_slices * M * Rp * 2);
    const auto rh = rsrc(l.t_hi, bytes), rl = rsrc(l.t_lo, bytes);
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = m0 + 16 * m + r, j = k0 + 32 * c + 8 * h;
        const uint32_t off = row < M && j < Rp ? (uint32_t)((q * M + row) * Rp + j) * 2 : kOob;
        t[0][m][c] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rh, off, 0, 0));
        t[1][m][c] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rl, off, 0, 0));
      }
  }
  // Of this lane's column of unit i: ranks of B in the eight from k0 + 32 c + 8 h on.
  __device__ __forceinline__ int ranks(int i, int c) const {
    const int n = first + 16 * at[i];
    return of[i] != 0 && n >= 0 && n < d ? max(0, min(8, ur[i] - (k0 + 32 * c + 8 * h))) : 0;
  }
  __device__ __forceinline__ void load_b() {
    const AdapterRef &ar = l.sl[q].ar;
    if (!ar.pooled) {
      const uint8_t *B = ar.B;
      const uint32_t R2 = ar.max_rank * 2, rows = (uint32_t)d * R2;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i > 0 && of[i] == 0) break;
        const auto rb = rsrc(B + (int64_t)us[i] * rows, rows);
        const uint32_t off = (uint32_t)(first + 16 * at[i]) * R2 + (k0 + 8 * h) * 2;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          b[i][c] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rb, ranks(i, c) > 0 ? off + 64 * c : kOob, 0, 0));
      }
      return;
    }
    // Lanes with no rank load the pool's first bytes.  Places in 16 bytes: all are below
    // 2^30 (256 ranks of 2^24 + 2^20 columns), so pages of 2^31 of them and more have
    // page 0 alone -- by a shift of 31, as one by 32 or more is taken modulo 32.
    const uint32_t k8 = (uint32_t)ar.k, shift = min(ar.page_shift - 4, 31), mask = (uint32_t)(ar.page_bytes >> 4) - 1;
    uint32_t off[kAhead][2];
    int32_t page[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t at16 = (uint32_t)ur[i] / 8 * (k8 + first + 16 * at[i]) + k0 / 8 + 4 * c + h;
        off[i][c] = ranks(i, c) > 0 ? at16 : 0;
        page[i][c] = ar.page_table[(int64_t)us[i] * ar.max_pages + (off[i][c] >> shift)];
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int64_t pg = ranks(i, c) > 0 ? page[i][c] : 0;
        b[i][c] = *reinterpret_cast<const u32x4_t *>(ar.pool + (pg << ar.page_shift) + (int64_t)(off[i][c] & mask) * 16);
      }
  }
  // The same where B's rows are no whole 16-byte vectors.
  __device__ __forceinline__ void load_b_by_rank() {
    const AdapterRef &ar = l.sl[q].ar;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        b[i][c] = u32x4_t{0, 0, 0, 0};
        const int n = ranks(i, c);
#pragma unroll 1
        for (int e = 0; e < n; ++e) {
          const uint32_t one = *reinterpret_cast<const uint16_t *>(
              adapter_b_ptr(ar, us[i], ur[i], first + 16 * at[i], k0 + 32 * c + 8 * h + e));
#pragma unroll
          for (int g = 0; g < 4; ++g) b[i][c][g] |= g == e >> 1 ? one << (16 * (e & 1)) : 0;
        }
      }
  }
  __device__ __forceinline__ void products(f32x4_t (&tot)[FM][FN]) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (of[i] == 0) return;
      if (ur[i] % 8 != 0 || l.sl[q].ar.pooled) {  // nothing past the rank
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int n = ranks(i, c);
#pragma unroll
          for (int e = 0; e < 4; ++e) b[i][c][e] = 2 * e + 1 < n ? b[i][c][e] : 2 * e < n ? b[i][c][e] & 0xFFFFu : 0u;
        }
      }
      const bool in = first + 16 * at[i] >= 0 && first + 16 * at[i] < d;
      const uint64_t to = of[i] >> (4 * h);
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, t[p][m][c]),
                                                          __builtin_bit_cast(bf16x8_t, b[i][c]), acc, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = in && (to >> (16 * m + e) & 1) ? acc[e] : 0.f;
#pragma unroll
        for (int jj = 0; jj < FN; ++jj)
          if (jj == at[i]) tot[m][jj] += acc;
      }
    }
  }
  // wave of lora_waves: every lora_waves-th unit, adapters in the order of their first
  // rows, columns inside.
  __device__ __forceinline__ void run(int wave, f32x4_t (&tot)[FM][FN]) {
    const int32_t *rows = l.row;
    own = of_row(rows, 0);
    const bool live = lane < ROWS && m0 + lane < M;
#pragma unroll 1
    for (q = 0; q < l.n_slices; ++q) {
      const SliceRef &sl = l.sl[q];
      d = (int)sl.d;
      first = n0 + r - (int)sl.col0;
      if (first - r >= d || first - r + 16 * FN <= 0) continue;
      lrank = of_row(rows, 1 + q);
#pragma unroll 1
      for (k0 = 0; k0 < sl.ar.max_rank; k0 += 64) {
        load_t();
        const bool has = live && own >= 0;
        uint64_t left = __ballot(has && lrank > k0), mine = 0;  // rows of adapters to come
        if (left == 0) break;
        // B's rows of whole 16-byte vectors, each of one page
        const bool vec = sl.ar.pooled ? __ballot(has && lrank % 8 != 0) == 0 : sl.ar.max_rank % 8 == 0;
        int s = 0, rk = 0, j = FN + wave;  // the unit's columns, FN more for each adapter to pass
#pragma unroll 1
        while (true) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            while (j >= FN && left != 0) {
              const int f = __builtin_ctzll(left);
              s = __builtin_amdgcn_readlane(own, f);
              rk = __builtin_amdgcn_readlane(lrank, f);
              mine = __ballot(own == s) & left;
              left &= ~mine;
              j -= FN;
            }
            of[i] = j < FN ? mine : 0;
            at[i] = j < FN ? j : 0;
            us[i] = s;
            ur[i] = rk;
            j += lora_waves<FM, FN>;
          }
          if (of[0] == 0) break;
          if (vec) load_b();
          else load_b_by_rank();
          products(tot);
          if (of[kAhead - 1] == 0) break;
        }
      }
    }
  }
};

// A workgroup takes 16 FM rows of x and 16 FN of W, each of its NW waves every
// NW-th record of k.  No wave shares an operand with another, so nothing waits
// but for its own loads, and the waves of a SIMD drift apart: one unpacks while
// the other multiplies.  W's records go straight to registers, x's rows by
// direct loads through the wave's own part of LDS (fragments read from memory
// would touch sixteen half lines an instruction: 54 cycles of a CU against 35),
// both PD records ahead.  The waves' sums meet in LDS at the end, in their order.
// Loads past the end of a wave's records, of x's rows and of its columns are
// past their buffer: they move nothing and give zeros.
//
// 1 x 9216 x 8192, groups of 128: 8.4 us, bound by W's bytes (4.7 TB/s, most of them from
// the last-level cache; 16 weights in turn, from HBM: 10.6, 3.75 TB/s); 7 x 4999 x 5000,
// groups of 32: 7.0, its records' latencies one after the other; 256 x 4096 x 4096: 16.0,
// unpacking and scaling between the products (matrix units busy 32%).  Eight waves a
// tile: sixteen took the same within 1%.
template <int FM, int FN, int NW, int PD, int SG, With kWith>
__global__ __launch_bounds__(64 * (NW + (kWith == kLora ? lora_waves<FM, FN> : 0))) void k_w4_split(W4GemmArgs p,
                                                                                              with_t<kWith> with) {
  constexpr int REC = (int)w4_record(SG), KS = 4 / SG;
  constexpr int HALF = FM * 2048, XI = 2 * FM;  // x: bytes of half a record, loads of 1 KiB
  constexpr int ALL = NW + (kWith == kLora ? lora_waves<FM, FN> : 0);
  constexpr int RING = NW * PD * 2 * HALF, PART = ALL * FM * FN * 1024;
  constexpr int kYounger = XI + (PD - 1) * (FN * (1 + SG) + 2 * XI) + FN * (1 + SG);
  constexpr int PLAN = kWith == kPlan ? (int)plan_detail::plan_sort_lds(plan_detail::kPlanRowBitsMax) : 0;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[std::max({RING, PART, PLAN})];
  int bx = blockIdx.x;
  if constexpr (kWith == kPlan) {
    if (bx == 0) {
      if (blockIdx.y == 0) plan_detail::plan_body<64 * NW>(with, smem, sizeof(smem));
      return;
    }
    --bx;
  } else if constexpr (kWith == kLora) {
    if (with.planned && bx == 0) {
      // by as many waves as it is made for; the others are gone before its barriers
      if (blockIdx.y == 0 && threadIdx.x < 64 * NW) plan_detail::plan_body<64 * NW>(with.plan, smem, sizeof(smem));
      return;
    }
    bx -= with.planned;
  }
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = bx * (16 * FN), m0 = blockIdx.y * (16 * FM);
  const int mr = min(16 * FM, p.M - m0), nr = min(16 * FN, p.N - n0);
  const uint32_t tile_bytes = (uint32_t)p.nb * REC;
  const auto rx = rsrc(p.x + (int64_t)m0 * p.ldx, (uint32_t)(((mr - 1) * p.ldx + p.K) * 2));
  const auto rw = rsrc(p.w + (int64_t)(n0 / 16) * tile_bytes, (uint32_t)((nr + 15) / 16) * tile_bytes);
  const int cnt = wave < p.nb ? (p.nb - 1 - wave) / NW + 1 : 0;  // this wave's records

  // x: eight rows a load, 128 bytes each; chunk c of row i stands at c ^ (i & 7)
  const int cx = ((lane & 7) ^ (lane >> 3)) * 8;
  const uint32_t vx = (uint32_t)((lane >> 3) * p.ldx * 2 + cx * 2), row8 = (uint32_t)(8 * p.ldx * 2);
  uint8_t *ring = smem + wave * (PD * 2 * HALF);
  auto load_x = [&](int t, int d, int u) {
    const int k0 = (wave + t * NW) * 128 + 64 * u;
    const uint32_t v = t < cnt && k0 + cx < p.K ? vx : kOob;
#pragma unroll
    for (int q = 0; q < XI; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rx, (__attribute__((address_space(3))) void *)(ring + (d * 2 + u) * HALF + q * 1024), 16, v,
          (uint32_t)k0 * 2 + q * row8, 0, 0);
  };
  u32x4_t wq[PD][FN];
  uint32_t sq[PD][FN][SG];
  auto load_w = [&](int t, int d) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const uint32_t at = t < cnt ? j * tile_bytes + (uint32_t)(wave + t * NW) * REC : kOob;
      wq[d][j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16, at, 0));
#pragma unroll
      for (int g = 0; g < SG; ++g)
        sq[d][j][g] = __builtin_amdgcn_raw_buffer_load_b32(rw, r * 4 + (int)kW4Codes + 64 * g, at, 0);
    }
  };
  f32x4_t tot[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int j = 0; j < FN; ++j) tot[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  const uint32_t xa = lds_addr(ring) + r * 128;
  if (kWith == kLora && wave >= NW) {
    if constexpr (kWith == kLora) {
      touch(with.lora);
      LoraPart<FM, FN>(with.lora, m0, n0).run(wave - NW, tot);
    }
  } else {
#pragma unroll
    for (int d = 0; d < PD; ++d) {
      load_w(d, d);
      asm volatile("" ::: "memory");
      load_x(d, d, 0);
      load_x(d, d, 1);
      asm volatile("" ::: "memory");
    }
    for (int t0 = 0; t0 < cnt; t0 += PD) {
#pragma unroll
      for (int d = 0; d < PD; ++d) {  // past the last record: zeros by zeros
        u32x4_t wc[FN];
        float s[FN][SG], z[FN][SG];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          wc[j] = wq[d][j];
#pragma unroll
          for (int g = 0; g < SG; ++g) {
            s[j][g] = scale_of(sq[d][j][g]);
            z[j][g] = (float)(sq[d][j][g] & 31u);
          }
        }
        load_w(t0 + d + PD, d);
        f32x4_t acc[FM][FN], sum[FM];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // Loads younger than this half's: the other half's of the same record or
          // the one before, W's and x's of the records between, W's just above.
          asm volatile("" ::: "memory");
          wait_vm<std::min(kYounger, 63)>();
          u32x4_t xf[2][FM];
          const uint32_t at = xa + (d * 2 + u) * HALF;
          read_half<FM>(at + (h ^ (r & 7)) * 16, at + ((4 + h) ^ (r & 7)) * 16, xf);
          load_x(t0 + d + PD, d, u);
          asm volatile("" ::: "memory");
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ks = 2 * u + i, g = ks / KS;
            const bool first = ks % KS == 0, last = ks % KS == KS - 1;
#pragma unroll
            for (int m = 0; m < FM; ++m)
              sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xf[i][m]), ones8(),
                                                               first ? zero : sum[m], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              const bf16x8_t wf = codes(wc[j][ks]);
#pragma unroll
              for (int m = 0; m < FM; ++m) {
                acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xf[i][m]), wf,
                                                                    first ? zero : acc[m][j], 0, 0, 0);
                if (last) {
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    tot[m][j][e] = __builtin_fmaf(s[j][g], __builtin_fmaf(-z[j][g], sum[m][e], acc[m][j][e]), tot[m][j][e]);
                }
              }
            }
          }
        }
      }
    }
  }
  wait_vm<0>();  // loads past the end have landed: LDS is free
  __syncthreads();
  f32x4_t(*part)[FM * FN][64] = reinterpret_cast<f32x4_t(*)[FM * FN][64]>(smem);
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int j = 0; j < FN; ++j) part[wave][m * FN + j][lane] = tot[m][j];
  __syncthreads();
  for (int u = wave; u < FM * FN; u += ALL) {
    f32x4_t v = part[0][u][lane];
#pragma unroll
    for (int q = 1; q < ALL; ++q) v += part[q][u][lane];
    const int n = n0 + u % FN * 16 + r, m = m0 + u / FN * 16 + 4 * h;
    if (n >= p.N) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m + e < p.M) p.y[(int64_t)(m + e) * p.ldy + n] = f32_to_bf16_bits(v[e]);
  }
}

template <int FM, int FN, int NW, int PD, int SG>
void launch_split(const W4GemmArgs &a, const PlanArgs *plan, hipStream_t st) {
  const dim3 grid((a.N + 16 * FN - 1) / (16 * FN) + (plan ? 1 : 0), (a.M + 16 * FM - 1) / (16 * FM)), block(64 * NW);
  if (plan) hipLaunchKernelGGL((k_w4_split<FM, FN, NW, PD, SG, kPlan>), grid, block, 0, st, a, *plan);
  else hipLaunchKernelGGL((k_w4_split<FM, FN, NW, PD, SG, kNone>), grid, block, 0, st, a, Nothing{});
}
template <int FM, int FN, int NW, int PD>
void launch_split(W4GemmArgs a, const PlanArgs *plan, hipStream_t st) {
  if (a.sg == 1) launch_split<FM, FN, NW, PD, 1>(a, plan, st);
  else if (a.sg == 2) launch_split<FM, FN, NW, PD, 2>(a, plan, st);
  else launch_split<FM, FN, NW, PD, 4>(a, plan, st);
}
template <int FM, int FN, int NW, int PD>
void launch_lora(const W4GemmArgs &a, const LoraWith &w, hipStream_t st) {
  const dim3 grid((a.N + 16 * FN - 1) / (16 * FN) + w.planned), block(64 * (NW + lora_waves<FM, FN>));
  if (a.sg == 1) hipLaunchKernelGGL((k_w4_split<FM, FN, NW, PD, 1, kLora>), grid, block, 0, st, a, w);
  else if (a.sg == 2) hipLaunchKernelGGL((k_w4_split<FM, FN, NW, PD, 2, kLora>), grid, block, 0, st, a, w);
  else hipLaunchKernelGGL((k_w4_split<FM, FN, NW, PD, 4, kLora>), grid, block, 0, st, a, w);
}

// Rows of x past 32-bit offsets of one another (the last tokens of long
// sequences, say): the same work with x by address, four waves a 16 x 16 tile.
template <int SG>
__global__ __launch_bounds__(256) void k_w4_far(W4GemmArgs p) {
  __shared__ f32x4_t part[3][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const uint16_t *x = p.x + (int64_t)min(m0 + (lane & 15), p.M - 1) * p.ldx;
  const uint8_t *w = p.w + (int64_t)blockIdx.x * p.nb * w4_record(SG);
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
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, codes(c[i]), acc, 0, 0, 0);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, ones8(), sum, 0, 0, 0);
      }
      const uint32_t sw = sc[g * 16];
      const float s = scale_of(sw), z = (float)(sw & 31u);
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

// ---------------------------------------------------------------- tiles
// More rows: WM x WN waves, each FM x FN products of 16 x 16, over BM rows of x
// and BN of W; KG times as many waves where a workgroup's records of k are
// shared out over KG groups, whose sums meet in LDS.  x goes through an LDS
// ring of ST stages (KG tiles of BM rows by 128 columns) by direct loads, W's
// records straight to the registers of the waves that unpack them, one
// stage ahead.
// W is rounded to bf16, s (q - z), before the product: scaling the groups' sums
// takes eight instructions for every 16 x 16 x group and as many sums again in
// registers, which tiles of this size have no room for.

// 16 bytes a lane from global memory straight into LDS, lane i's at lds + 16 i
// (as in gemm_mx.hip: asm, because the compiler would drain every load ahead
// of each LDS read; the waits are explicit; no register output).
__device__ __forceinline__ void dma(i32x4_t r, uint32_t lds, uint32_t off, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               : : "s"(lds), "v"(off), "s"(r), "s"(soff));
}
__device__ __forceinline__ i32x4_t rsrc_words(const void *p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
                 __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// Waits for this wave's LDS accesses but not for its loads.
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Eight weights s (q - z), rounded to bf16 once each: s of 19 bits times z or
// q - z of five is exact.
__device__ __forceinline__ bf16x8_t weights(uint32_t w, float s, float sz) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  f32x2_t v[4];
  v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.f, false);
  v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.f, true);
  v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.f, false);
  v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.f, true);
  u32x4_t o;
#pragma unroll
  for (int p = 0; p < 4; ++p) o[p] = pack_bf16x2(__builtin_fmaf(s, v[p][0], -sz), __builtin_fmaf(s, v[p][1], -sz));
  return __builtin_bit_cast(bf16x8_t, o);
}

template <int FM, int FN, int WM, int WN, int KG, int ST, int WS, int SG>
struct WTile {
  static constexpr int NW = WM * WN * KG, NT = 64 * NW;
  static constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  static constexpr int XSTAGE = KG * BM * 128;
  static constexpr int TILES = KG * BN / 16, SB = (TILES + 15) / 16;  // records a stage of W, KiB of its scales a group
  static constexpr int WSTAGE = TILES * 1024 + SG * SB * 1024;
  // 1 KiB loads a stage, and a wave's (where there are fewer than waves,
  // several load the same)
  static constexpr int XI = XSTAGE / 1024, XL = (XI + NW - 1) / NW;
  static constexpr int WI = WSTAGE / 1024, WL = (WI + NW - 1) / NW;
  static constexpr int W0 = ST * XSTAGE;
  static constexpr int CLD = BN + 8;
  static constexpr int PART = (KG - 1) * BM * BN * 4;
  static constexpr int SMEM = std::max(W0 + WS * WSTAGE, std::max(PART, BM * CLD * 2));
  static_assert(SMEM <= 160 * 1024, "LDS");
  static_assert(XSTAGE % 1024 == 0 && ST >= 3 && WS >= 2, "stages");
  static_assert((ST - 1) * XL + ST / 2 * WL < 64, "vmcnt");
};

// 8192 x 4096 x 4096 (groups of 64, 256 x 256 tiles): 233 us, 1.18 PFLOP/s, against 202
// at the library's bf16 rate; 512 x 9216 x 8192 (groups of 128, 128 x 160): 85 - 95.  Unpacking
// bounds both: it takes issue slots that other waves' matrix instructions do not
// fill (two VALU instructions behind one are free, a third takes a quarter of it more).
//
// The tile of this workgroup: each XCD takes a contiguous run of tiles, bands
// of eight row tiles down, then across.
__device__ __forceinline__ void tile_of(const W4GemmArgs &p, uint32_t b, int &tm, int &tn) {
  const uint32_t nblk = (uint32_t)p.tiles_m * p.tiles_n;
  const uint32_t xcd = b & 7, each = nblk >> 3, more = nblk & 7;
  const uint32_t t = xcd * each + (xcd < more ? xcd : more) + (b >> 3);
  const uint32_t band = t / (8u * p.tiles_n), in = t - band * 8u * p.tiles_n;
  const uint32_t rows_in = min(8u, (uint32_t)p.tiles_m - band * 8u);
  tm = (int)(band * 8u + in % rows_in);
  tn = (int)(in / rows_in);
}

template <int FM, int FN, int WM, int WN, int KG, int ST, int WS, int SG, With kWith>
__global__ __launch_bounds__(64 * WM * WN * KG) void k_w4_tile(W4GemmArgs p, with_t<kWith> with) {
  using T = WTile<FM, FN, WM, WN, KG, ST, WS, SG>;
  constexpr int BM = T::BM, BN = T::BN, REC = (int)w4_record(SG);
  static_assert(T::SMEM >= plan_detail::plan_sort_lds(plan_detail::kPlanRowBitsMax), "room for the plan");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::SMEM];
  uint32_t b = blockIdx.x;
  if constexpr (kWith == kPlan) {
    if (b == 0) {
      plan_detail::plan_body<T::NT>(with, smem, sizeof(smem));
      return;
    }
    --b;
  }
  int tm, tn;
  tile_of(p, b, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG == 1 ? 0 : wave / (WM * WN), wt = KG == 1 ? wave : wave % (WM * WN);
  const int wm0 = wt / WN * (16 * FM), wn0 = wt % WN * (16 * FN);
  const int mr = min(BM, p.M - m0), nr = min(BN, p.N - n0);
  const int nk = (p.nb + KG - 1) / KG;
  const uint32_t tile_bytes = (uint32_t)p.nb * REC;  // of 16 rows of W
  i32x4_t rx = rsrc_words(p.x + (int64_t)m0 * p.ldx, (uint32_t)(((mr - 1) * p.ldx + p.K) * 2));
  i32x4_t rw = rsrc_words(p.w + (int64_t)(n0 / 16) * tile_bytes, (uint32_t)((nr + 15) / 16) * tile_bytes);
  asm volatile("s_nop 4" : "+s"(rx), "+s"(rw));
  const uint32_t base = __builtin_amdgcn_readfirstlane(lds_addr(smem));

  // x: eight rows a load, 128 bytes each; chunk c of row i stands at c ^ (i & 7)
  uint32_t vx[T::XL];
  int cx[T::XL];
#pragma unroll
  for (int i = 0; i < T::XL; ++i) {
    const int ins = (wave * T::XL + i) % T::XI, row = ins % (BM / 8) * 8 + (lane >> 3);
    cx[i] = ((lane & 7) ^ (lane >> 3)) * 8 + ins / (BM / 8) * 128;
    vx[i] = (uint32_t)((row * p.ldx + cx[i]) * 2);
  }
  auto load_x = [&](int i, int u) {  // of half record u
    const int k0 = (u >> 1) * (KG * 128) + (u & 1) * 64;
    dma(rx, base + u % ST * T::XSTAGE + (wave * T::XL + i) % T::XI * 1024, k0 + cx[i] < p.K ? vx[i] : kOob,
        (uint32_t)k0 * 2);
  };
  // W: the records' codes, a load each, then their scales, sixteen records a
  // load; those of records past the last one are zero
  auto load_w = [&](int i, int kt) {
    const int ins = (wave * T::WL + i) % T::WI;
    const uint32_t to = base + T::W0 + kt % WS * T::WSTAGE + ins * 1024;
    if (ins < T::TILES) {
      const int q = KG == 1 ? 0 : ins / (BN / 16), blk = kt * KG + q;
      dma(rw, to, blk < p.nb ? lane * 16 : kOob, (uint32_t)(ins - q * (BN / 16)) * tile_bytes + (uint32_t)blk * REC);
    } else {
      const int g = (ins - T::TILES) / T::SB, t = (ins - T::TILES) % T::SB * 16 + (lane >> 2);
      const int q = KG == 1 ? 0 : t / (BN / 16), blk = kt * KG + q;
      const uint32_t v = (uint32_t)(t - q * (BN / 16)) * tile_bytes + (uint32_t)blk * REC + (lane & 3) * 16;
      dma(rw, to, t < T::TILES && blk < p.nb ? v : kOob, (uint32_t)(kW4Codes + 64 * g));
    }
  };
  f32x4_t tot[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) tot[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const uint8_t *xb = smem + (kg * BM + wm0 + r) * 128;
  const uint8_t *wb = smem + T::W0 + (kg * (BN / 16) + wn0 / 16) * 1024 + lane * 16;
  // Half record s = 2 kt + u is multiplied while the rows of x of half record s +
  // ST - 1 and, with the even ones, the record kt + WS - 1 of W are loaded, in
  // that order; the prologue issues what the halves before the first would have.
#pragma unroll
  for (int kt = 0; kt < WS - 1; ++kt) {
    if (2 * (WS - 1 - kt) < ST) continue;
#pragma unroll
    for (int i = 0; i < T::WL; ++i) load_w(i, kt);
  }
#pragma unroll
  for (int s = 1 - ST; s < 0; ++s) {
#pragma unroll
    for (int i = 0; i < T::XL; ++i) load_x(i, s + ST - 1);
    if (s % 2 == 0) {
#pragma unroll
      for (int i = 0; i < T::WL; ++i) load_w(i, s / 2 + WS - 1);
    }
  }
  // Loads that may be on their way when half record s starts: those of the ST - 2
  // halves before it -- of the even ones, which turn to another record of W, of
  // no more than came after that.
  constexpr int n0h = std::min(ST - 2, 2 * WS - 3), n1h = ST - 2;
  constexpr int kWait0 = n0h * T::XL + n0h / 2 * T::WL, kWait1 = n1h * T::XL + (n1h + 1) / 2 * T::WL;
  uint32_t stage = 0;
  for (int kt = 0; kt < nk; ++kt) {
    u32x4_t wc[FN];
    float sc[FN][SG], zc[FN][SG];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 0) wait_vm<kWait0>();
      else wait_vm<kWait1>();
      barrier();  // every wave's have, and the stage before is free
      if (u == 0) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          wc[j] = *reinterpret_cast<const u32x4_t *>(wb + kt % WS * T::WSTAGE + j * 1024);
#pragma unroll
          for (int g = 0; g < SG; ++g) {
            const int t = kg * (BN / 16) + wn0 / 16 + j;
            const uint32_t sw = *reinterpret_cast<const uint32_t *>(
                smem + T::W0 + kt % WS * T::WSTAGE + (T::TILES + g * T::SB) * 1024 + t * 64 + r * 4);
            sc[j][g] = scale_of(sw);
            zc[j][g] = sc[j][g] * (float)(sw & 31u);
          }
        }
      }
      const int un = 2 * kt + u + ST - 1;  // the half record to load
      constexpr int nl = T::XL + T::WL;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ks = 2 * u + i, g = ks * SG / 4;
        bf16x8_t wf[FN], xf[FM];
#pragma unroll
        for (int m = 0; m < FM; ++m)
          xf[m] = *reinterpret_cast<const bf16x8_t *>(xb + stage * T::XSTAGE + m * 2048 + ((i * 4 + h) ^ (r & 7)) * 16);
        // half of the loads with each step
#pragma unroll
        for (int d = i * nl / 2; d < (i + 1) * nl / 2; ++d) {
          if (d < T::XL) load_x(d, un);
          else if (u == 0) load_w(d - T::XL, kt + WS - 1);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) wf[j] = weights(wc[j][ks], sc[j][g], zc[j][g]);
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int m = 0; m < FM; ++m)
            tot[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[j], xf[m], tot[m][j], 0, 0, 0);
      }
      stage = stage + 1 == ST ? 0 : stage + 1;
    }
  }
  wait_vm<0>();  // the loads past the end have landed: LDS is free

  if constexpr (KG > 1) {  // the groups' sums, in the groups' order
    __syncthreads();
    f32x4_t *part = reinterpret_cast<f32x4_t *>(smem);
    auto at = [&](int q, int i, int j) { return (((q - 1) * WM * WN + wt) * FM * FN + i * FN + j) * 64 + lane; };
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) part[at(kg, i, j)] = tot[i][j];
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 1; q < KG; ++q) tot[i][j] += part[at(q, i, j)];
    }
  }
  __syncthreads();
  // rounded once and stored, through LDS, as whole rows of 16-byte vectors
  uint16_t *ct = reinterpret_cast<uint16_t *>(smem);
  if (kg == 0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        // lane: row r of x, columns 4 h + e
        *reinterpret_cast<uint2 *>(ct + (wm0 + i * 16 + r) * T::CLD + wn0 + j * 16 + 4 * h) =
            make_uint2(pack_bf16x2(tot[i][j][0], tot[i][j][1]), pack_bf16x2(tot[i][j][2], tot[i][j][3]));
      }
  }
  __syncthreads();
  constexpr int CPR = BN / 8;
  for (int c = threadIdx.x; c < BM * CPR; c += T::NT) {
    const int row = c / CPR, col = (c - row * CPR) * 8;
    if (row >= mr || col >= nr) continue;
    const uint16_t *src = ct + row * T::CLD + col;
    uint16_t *dst = p.y + (int64_t)(m0 + row) * p.ldy + n0 + col;
    if (col + 8 <= nr) {
      const uint4 v = *reinterpret_cast<const uint4 *>(src);
      __builtin_memcpy(dst, &v, 16);  // any alignment
    } else {
      for (int e = 0; e < 8 && col + e < nr; ++e) dst[e] = src[e];
    }
  }
}

template <int FM, int FN, int WM, int WN, int KG, int ST, int WS, int SG>
void launch_tile(const W4GemmArgs &a, const PlanArgs *plan, hipStream_t st) {
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_n) + (plan ? 1 : 0)), block(64 * WM * WN * KG);
  if (plan) hipLaunchKernelGGL((k_w4_tile<FM, FN, WM, WN, KG, ST, WS, SG, kPlan>), grid, block, 0, st, a, *plan);
  else hipLaunchKernelGGL((k_w4_tile<FM, FN, WM, WN, KG, ST, WS, SG, kNone>), grid, block, 0, st, a, Nothing{});
}
template <int FM, int FN, int WM, int WN, int KG, int ST, int WS>
void launch_tile(W4GemmArgs a, const PlanArgs *plan, hipStream_t st) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + BN - 1) / BN;
  if (a.sg == 1) launch_tile<FM, FN, WM, WN, KG, ST, WS, 1>(a, plan, st);
  else if (a.sg == 2) launch_tile<FM, FN, WM, WN, KG, ST, WS, 2>(a, plan, st);
  else launch_tile<FM, FN, WM, WN, KG, ST, WS, 4>(a, plan, st);
}

// ---------------------------------------------------------------- which
// With t tiles over the 256 CUs, of which a CU holds `fit` at once, and records
// of 128 columns, a shape's time is taken as
//   s + ceil(t / 256 fit) (e + c records) + (ceil(t / 256) w + t / 256 f) records
// in us: what a round of workgroups takes alone, what those that share a CU
// and those on other CUs add.  The numbers are least-squares fits (none
// negative) of each shape's times at up to 189 sizes with groups of 128, 64 and
// 32 (M from 1 to 8192, d x k of 9216 x 8192, 4096 x 4096, 5120 x 5120, 1024 x
// 4096, 1024 x 1024, 1024 x 8192, 512 x 2048, 4096 x 512 and 8192 x 1024), good to
// 3 - 12%; the choice takes 1.03 of the best of 25 shapes' time, on the mean.
// The table holds those without which that gets worse by 0.1% or more.
struct Cost {
  int fit;
  float s, e, c, w, f;
};
struct Shape {
  int bm, bn;
  bool rounds;  // the weights, to bf16
  int held;     // workgroups that a CU holds
  Cost cost[3];  // groups of 128 and more, 64, 32
  void (*launch)(W4GemmArgs, const PlanArgs *, hipStream_t);
};
constexpr int held(int smem, int waves) { return std::max(1, std::min(160 * 1024 / smem, 16 / waves)); }
template <int FM, int FN, int NW, int PD>
constexpr Shape split(Cost g128, Cost g64, Cost g32) {
  return {16 * FM, 16 * FN, false, held(std::max(NW * PD * FM * 4096, NW * FM * FN * 1024), NW),
          {g128, g64, g32}, launch_split<FM, FN, NW, PD>};
}
template <int FM, int FN, int WM, int WN, int KG, int ST, int WS>
constexpr Shape tile(Cost c) {
  return {16 * FM * WM, 16 * FN * WN, true, held(WTile<FM, FN, WM, WN, KG, ST, WS, 1>::SMEM, WM * WN * KG),
          {c, c, c}, launch_tile<FM, FN, WM, WN, KG, ST, WS>};
}
const Shape kShapes[] = {
    split<1, 1, 8, 2>({1, 2.57f, 0.872f, 0.0337f, 0.f, 0.014f},
                     {1, 2.6f, 0.93f, 0.0404f, 0.f, 0.0111f},
                     {1, 2.45f, 0.988f, 0.0472f, 0.f, 0.0113f}),
    split<1, 3, 8, 1>({2, 2.35f, 1.15f, 0.f, 0.0636f, 0.047f},
                     {2, 2.f, 1.48f, 0.0035f, 0.0922f, 0.0322f},
                     {2, 2.08f, 1.2f, 0.031f, 0.114f, 0.0278f}),
    split<1, 2, 8, 1>({4, 1.49f, 1.96f, 0.f, 0.0411f, 0.0302f},
                     {2, 2.54f, 0.854f, 0.f, 0.0535f, 0.0244f},
                     {2, 2.08f, 1.27f, 0.0147f, 0.074f, 0.0207f}),
    split<2, 2, 8, 1>({1, 2.7f, 0.671f, 0.0782f, 0.f, 0.0368f},
                     {1, 2.6f, 0.75f, 0.0883f, 0.f, 0.0372f},
                     {1, 2.74f, 0.711f, 0.136f, 0.f, 0.0148f}),
    split<2, 3, 8, 1>({1, 2.51f, 0.831f, 0.118f, 0.f, 0.0413f},
                     {1, 2.47f, 0.875f, 0.15f, 0.f, 0.0362f},
                     {1, 1.54f, 1.88f, 0.192f, 0.f, 0.0617f}),
    split<2, 4, 8, 1>({1, 1.63f, 1.7f, 0.139f, 0.f, 0.0604f},
                     {1, 1.51f, 1.87f, 0.186f, 0.f, 0.0695f},
                     {1, 1.58f, 2.04f, 0.253f, 0.f, 0.0595f}),
    split<4, 3, 8, 1>({1, 1.09f, 3.03f, 0.186f, 0.f, 0.0754f},
                     {1, 1.04f, 2.96f, 0.225f, 0.f, 0.0779f},
                     {1, 1.28f, 3.18f, 0.317f, 0.f, 0.0752f}),
    split<4, 4, 8, 1>({1, 1.34f, 3.2f, 0.27f, 0.f, 0.103f},
                     {1, 1.48f, 3.12f, 0.295f, 0.f, 0.105f},
                     {1, 1.37f, 3.57f, 0.396f, 0.f, 0.0956f}),
    tile<4, 2, 1, 4, 2, 4, 2>({1, 1.48f, 2.4f, 0.582f, 0.f, 0.101f}),
    tile<8, 2, 1, 4, 2, 3, 2>({1, 2.19f, 2.74f, 0.789f, 0.f, 0.242f}),
    tile<4, 5, 2, 2, 2, 3, 2>({1, 1.97f, 3.25f, 1.17f, 0.f, 0.272f}),
    tile<8, 2, 2, 4, 1, 4, 2>({1, 0.f, 5.06f, 1.51f, 0.f, 0.481f}),
    tile<8, 3, 2, 4, 1, 3, 2>({1, 0.547f, 4.89f, 2.06f, 0.f, 0.547f}),
    tile<8, 4, 2, 4, 1, 3, 2>({1, 0.f, 6.5f, 2.68f, 0.f, 0.733f}),
};

// A shape's time by the model above.
double time_of(const Cost &c, int64_t tiles, int32_t nb) {
  const double rounds = (double)((tiles + 256 * c.fit - 1) / (256 * c.fit)), cu = (double)((tiles + 255) / 256);
  return c.s + rounds * (c.e + (double)c.c * nb) + (cu * c.w + (double)tiles / 256 * c.f) * nb;
}

// slabs whose grids stay far below what a launch takes
constexpr int64_t kSlabM = int64_t(1) << 18, kSlabN = int64_t(1) << 20;

// The shape that takes least of those that round the weights, or of the others.
const Shape &best_of(int64_t M, int64_t N, int32_t nb, int32_t sg, bool rounds, double *time) {
  const Shape *best = nullptr;
  for (const Shape &h : kShapes) {
    if (h.rounds != rounds) continue;
    const double t = time_of(h.cost[sg >> 1], (M + h.bm - 1) / h.bm * ((N + h.bn - 1) / h.bn), nb);
    if (best == nullptr || t < *time) {
      best = &h;
      *time = t;
    }
  }
  return *best;
}

// The rows from which on a product over a weight of these sizes rounds the weights:
// the first number at which that is faster by the model, though with a few more it
// may not be, so that what a row's values are rounded to does not go back and forth
// with the rows beside it.  Never up to kW4Rows, which the layer's own shapes take.
// Sought in steps of the smallest tile's rows, past 512 in steps of 1/16, once for
// sizes that are not among a thread's last 16 (5 us; else as long as one shape's time).
// Next to the faster of both everywhere, at 19 weights and 33 to 8192 rows: 1.0001
// of the time by the model on the mean, 1.08 at most.  Measured where it decides, groups
// of 128: 9216 x 8192, 193 rows 58.5 us against 53.1, 256 rows 59.2 against 60.1; 5120 x
// 5120, 400 rows 38.4 against 42.7; 1024 x 8192, 2100 rows 60.3 against 62.5.
int64_t rounded_from(int64_t N, int32_t nb, int32_t sg) {
  struct Seen {
    int64_t N;
    int32_t nb, sg;
    int64_t from;
  };
  thread_local Seen seen[16];
  Seen &e = seen[(N / 16 + 5 * nb + sg) % 16];
  if (e.N != N || e.nb != nb || e.sg != sg) {
    int64_t m = kW4Rows + 1;
    for (; m <= kSlabM; m += std::max<int64_t>(16, m / 256 * 16)) {
      double exact, rounded;
      best_of(m, N, nb, sg, false, &exact);
      best_of(m, N, nb, sg, true, &rounded);
      if (rounded < exact) break;
    }
    e = Seen{N, nb, sg, m <= kSlabM ? m : INT64_MAX};
  }
  return e.from;
}

const Shape &best_of(int64_t M, int64_t N, int32_t nb, int32_t sg) {
  double t;
  return best_of(M, N, nb, sg, M >= rounded_from(N, nb, sg), &t);
}

// The same with the adapters' part, which leaves a CU room for one workgroup.  Every
// row has the sums that the shapes above give it.  Fits of the whole layer's times at
// 1 to 32 rows, ranks 16 and 64, d x k of 32768 x 8192, 32768 x 4096, 20480 x 2048,
// 16384 x 4096, 10240 x 8192 and below, good to 6 - 15% (ranks and adapters are not
// in them); the choice takes 1.02 of the best of ten shapes' time, on the mean.
struct LoraShape {
  int bm, bn;
  Cost cost[3];
  void (*launch)(const W4GemmArgs &, const LoraWith &, hipStream_t);
};
template <int FM, int FN, int NW, int PD>
constexpr LoraShape lora(Cost g128, Cost g64, Cost g32) {
  return {16 * FM, 16 * FN, {g128, g64, g32}, launch_lora<FM, FN, NW, PD>};
}
const LoraShape kLoraShapes[] = {
    lora<1, 1, 8, 2>({1, 9.8f, 2.71f, 0.f, 0.f, 0.0372f},
                     {1, 9.95f, 2.64f, 0.f, 0.f, 0.0435f},
                     {1, 10.1f, 2.58f, 0.f, 0.f, 0.0497f}),
    lora<1, 2, 8, 1>({1, 10.2f, 1.61f, 0.0062f, 0.f, 0.0759f},
                     {1, 9.54f, 1.65f, 0.0286f, 0.f, 0.071f},
                     {1, 8.87f, 1.68f, 0.051f, 0.f, 0.0662f}),
    lora<1, 3, 8, 1>({1, 7.78f, 2.74f, 0.056f, 0.f, 0.0396f},
                     {1, 7.59f, 2.37f, 0.0918f, 0.f, 0.0387f},
                     {1, 7.4f, 2.f, 0.128f, 0.f, 0.0377f}),
    lora<1, 4, 8, 1>({1, 7.12f, 6.04f, 0.0324f, 0.f, 0.0594f},
                     {1, 8.35f, 4.16f, 0.0764f, 0.f, 0.0954f},
                     {1, 9.57f, 2.27f, 0.12f, 0.f, 0.131f}),
    lora<2, 2, 8, 1>({1, 7.62f, 5.67f, 0.0455f, 0.f, 0.0573f},
                     {1, 7.51f, 5.54f, 0.0705f, 0.f, 0.0506f},
                     {1, 7.4f, 5.4f, 0.0954f, 0.f, 0.0439f}),
    lora<2, 3, 8, 1>({1, 8.36f, 6.28f, 0.064f, 0.f, 0.0595f},
                     {1, 8.57f, 5.7f, 0.102f, 0.f, 0.0601f},
                     {1, 8.79f, 5.12f, 0.14f, 0.f, 0.0607f}),
    lora<2, 4, 8, 1>({1, 9.26f, 7.45f, 0.0585f, 0.f, 0.12f},
                     {1, 8.9f, 7.35f, 0.105f, 0.f, 0.12f},
                     {1, 8.55f, 7.26f, 0.151f, 0.f, 0.12f}),
};
const LoraShape &best_lora(int64_t M, int64_t N, int32_t nb, int32_t sg) {
  const LoraShape *best = nullptr;
  double least = 0;
  for (const LoraShape &h : kLoraShapes) {
    if (h.bm != (M > 16 ? 32 : 16)) continue;  // W once
    const double t = time_of(h.cost[sg >> 1], (N + h.bn - 1) / h.bn, nb);
    if (best == nullptr || t < least) {
      best = &h;
      least = t;
    }
  }
  return *best;
}
static_assert(kW4Rows == 32, "the rows of a tile");

}  // namespace

// A grid of 2^32 threads or more is cut off without an error: slabs of rows that
// hold at most this many records (a row of records, 2^17 at most, always fits).
static constexpr int64_t kSlabRecords = int64_t(1) << 22;

hipError_t launch_w4_pack(const W4Args &all, hipStream_t st) {
  const int64_t slab = kSlabRecords / all.nb * 16;
  for (int64_t n0 = 0; n0 < all.d; n0 += slab) {
    W4Args a = all;
    a.d = std::min(slab, all.d - n0);
    a.q += n0 * a.ldq;
    a.scales = (const uint8_t *)a.scales + n0 * a.lds * (a.scale_dtype == 1 ? 2 : 4);
    if (a.zeros) a.zeros += n0 * a.ldz;
    a.w += n0 / 16 * a.nb * w4_record(a.sg);
    hipLaunchKernelGGL(k_w4_pack, dim3((unsigned)((a.d + 15) / 16 * a.nb)), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_w4_dequantize(const W4Args &all, hipStream_t st) {
  const int32_t per_row = (all.nb + kDqRecords - 1) / kDqRecords;
  const int64_t slab = kSlabRecords / per_row * 16;
  for (int64_t n0 = 0; n0 < all.d; n0 += slab) {
    W4Args a = all;
    a.d = std::min(slab, all.d - n0);
    a.w += n0 / 16 * a.nb * w4_record(a.sg);
    a.y = (uint8_t *)a.y + n0 * a.ldy * (a.dtype == 1 ? 2 : 4);
    const dim3 grid((unsigned)((a.d + 15) / 16 * per_row));
    if (a.dtype == 1) hipLaunchKernelGGL(k_w4_dequantize<uint16_t>, grid, dim3(256), 0, st, a, per_row);
    else hipLaunchKernelGGL(k_w4_dequantize<float>, grid, dim3(256), 0, st, a, per_row);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int gemm_w4_shape(int64_t M, int64_t k, int64_t d, int32_t sg, int32_t out[3]) {
  const Shape &s = best_of(std::min(M, kSlabM), std::min(d, kSlabN), (int32_t)((k + 127) / 128), sg);
  out[0] = s.bm;
  out[1] = s.bn;
  out[2] = s.rounds;
  return (int)(&s - kShapes);
}

// rows of x of a tile past 32-bit offsets of one another
static bool far_rows(const W4GemmArgs &a) { return (uint64_t)256 * a.ldx * 2 + (uint64_t)a.K * 2 >= kOob; }

bool gemm_w4_adds_lora(const W4GemmArgs &a) { return a.M <= kW4Rows && a.N <= kSlabN && !far_rows(a); }

// Where the CUs are not all full of tiles to the last, a plan costs no more than
// its own time.
bool gemm_w4_runs_plan(const W4GemmArgs &a) {
  if (a.M > kPlanMaxRows || a.N > kSlabN || far_rows(a)) return false;
  const Shape &h = best_of(a.M, a.N, a.nb, a.sg);
  const int64_t tiles = (int64_t)((a.M + h.bm - 1) / h.bm) * ((a.N + h.bn - 1) / h.bn);
  return tiles % (256 * h.held) != 0;
}
bool gemm_w4_lora_runs_plan(const W4GemmArgs &a) {
  const int bn = best_lora(a.M, a.N, a.nb, a.sg).bn;
  return (a.N + bn - 1) / bn % 256 != 0;
}

int linear_w4_shape(const W4GemmArgs &a, int32_t out[3]) {
  constexpr int kFew = sizeof(kLoraShapes) / sizeof(kLoraShapes[0]);
  if (!gemm_w4_adds_lora(a)) {
    const int i = gemm_w4_shape(a.M, a.K, a.N, a.sg, out);
    out[2] = gemm_w4_runs_plan(a);
    return kFew + i;
  }
  const LoraShape &s = best_lora(a.M, a.N, a.nb, a.sg);
  out[0] = s.bm;
  out[1] = s.bn;
  out[2] = gemm_w4_lora_runs_plan(a);
  return (int)(&s - kLoraShapes);
}

hipError_t launch_gemm_w4_lora(const W4GemmArgs &a, const W4Lora &l, hipStream_t st, const PlanArgs *plan) {
  if (!gemm_w4_adds_lora(a)) return hipErrorInvalidValue;
  LoraWith w{l, {}, plan != nullptr};
  if (plan) w.plan = *plan;
  best_lora(a.M, a.N, a.nb, a.sg).launch(a, w, st);
  return hipGetLastError();
}

hipError_t launch_gemm_w4(const W4GemmArgs &all, hipStream_t st, const PlanArgs *plan) {
  const bool far = far_rows(all);
  if (plan && !gemm_w4_runs_plan(all)) return hipErrorInvalidValue;
  // all slabs alike
  const bool rounds = all.M >= rounded_from(std::min<int64_t>(all.N, kSlabN), all.nb, all.sg);
  for (int64_t m0 = 0; m0 < all.M; m0 += kSlabM)
    for (int64_t n0 = 0; n0 < all.N; n0 += kSlabN) {
      W4GemmArgs a = all;
      a.M = (int32_t)std::min(kSlabM, all.M - m0);
      a.N = (int32_t)std::min(kSlabN, all.N - n0);
      a.x += m0 * a.ldx;
      a.w += n0 / 16 * a.nb * w4_record(a.sg);
      a.y += m0 * a.ldy + n0;
      if (!far) {
        double t;
        best_of(a.M, a.N, a.nb, a.sg, rounds, &t).launch(a, plan, st);
      } else {
        const dim3 grid((a.N + 15) / 16, (a.M + 15) / 16);
        if (a.sg == 1) hipLaunchKernelGGL(k_w4_far<1>, grid, dim3(256), 0, st, a);
        else if (a.sg == 2) hipLaunchKernelGGL(k_w4_far<2>, grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL(k_w4_far<4>, grid, dim3(256), 0, st, a);
      }
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace lora
