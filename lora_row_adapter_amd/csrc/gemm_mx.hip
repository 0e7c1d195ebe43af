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
#include <algorithm>
#include <type_traits>

#include "mx_device.hpp"

namespace lora {

using namespace mx;

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr uint32_t kOob = 0xFFFFFFF0u;  // past every buffer: loads give zeros

// a 4-bit operand takes the lower half of the instruction's registers
__device__ __forceinline__ i32x8_t widen(i32x4_t v) {
  return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
}
__device__ __forceinline__ i32x8_t widen(i32x8_t v) { return v; }
template <int XF>
using frag_t = std::conditional_t<XF == kFp8, i32x8_t, i32x4_t>;
__device__ __forceinline__ i32x8_t frag8(i32x4_t a, i32x4_t b) {
  return i32x8_t{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// acc += W fragment (fp4, rows of the result) x x fragment (columns)
template <int XF>
__device__ __forceinline__ f32x4_t mfma(i32x4_t w, frag_t<XF> x, f32x4_t acc, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w), widen(x), acc, 4, XF == kFp8 ? 0 : 4, 0,
                                                          (int)sw, 0, (int)sx);
}

// ---------------------------------------------------------------------------
// Tiles through LDS.
// ---------------------------------------------------------------------------

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// 16 bytes a lane from global memory straight into LDS, lane i's at lds +
// 16 i.  Written as asm because the compiler, which cannot tell ring stages
// apart, would drain every load in flight before each LDS read; the waits are
// explicit (wait_vm, then a barrier, which the compiler moves no LDS access
// over).  It has no register output, so nothing is reused before it lands,
// and nothing else in these kernels uses m0, from whose write the s_nop keeps
// the load.
// The range check takes `off` + `soff` without wrapping, dword by dword
// (checked on the device), so lanes at kOob and rows past a tile's last load
// zeros.
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
// The four descriptors, and the distance that their first loads keep from
// the vector instructions that wrote scalar registers.
struct Sources {
  i32x4_t x, w, xs, ws;
};
// Each ends with its last row's blocks (of scales: with the four that share a
// dword), whatever the stride.
template <int XF>
__device__ __forceinline__ Sources sources(const MxGemmArgs &p, int m0, int n0, int mr, int nr) {
  const int64_t sb = (p.nb + 3) & ~3;
  const int64_t xb = (int64_t)p.nb * (XF == kFp8 ? 32 : 16), wb = (int64_t)p.nb * 16;
  Sources s = {rsrc_words(p.x + (int64_t)m0 * p.ldx, (uint32_t)((mr - 1) * p.ldx + xb)),
               rsrc_words(p.w + (int64_t)n0 * p.ldw, (uint32_t)((nr - 1) * p.ldw + wb)),
               rsrc_words(p.xs + (int64_t)m0 * p.ldxs, (uint32_t)((mr - 1) * p.ldxs + sb)),
               rsrc_words(p.wsc + (int64_t)n0 * p.ldws, (uint32_t)((nr - 1) * p.ldws + sb))};
  asm volatile("s_nop 4" : "+s"(s.x), "+s"(s.w), "+s"(s.xs), "+s"(s.ws));
  return s;
}
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p);
}

// The tile of this workgroup.  Workgroups go round the eight XCDs: each XCD
// takes a contiguous run of tiles (its own L2), bands of eight row tiles
// down, then across.
__device__ __forceinline__ void tile_of(const MxGemmArgs &p, int &tm, int &tn) {
  const uint32_t nblk = (uint32_t)p.tiles_m * p.tiles_n, b = blockIdx.x;
  const uint32_t xcd = b & 7, each = nblk >> 3, more = nblk & 7;
  const uint32_t t = xcd * each + (xcd < more ? xcd : more) + (b >> 3);
  const uint32_t band = t / (8u * p.tiles_n), in = t - band * 8u * p.tiles_n;
  const uint32_t rows_in = min(8u, (uint32_t)p.tiles_m - band * 8u);
  tm = (int)(band * 8u + in % rows_in);
  tn = (int)(in / rows_in);
}

// A barrier that waits for this wave's LDS accesses but not for its loads (a
// fenced one would drain the ring); LDS accesses stay on their side of it.
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Rounds the sums once and stores them, through LDS, as whole rows of
// 16-byte vectors.  has: whether this wave holds a part of the tile.
template <int BM, int BN, int FM, int FN, int NT>
__device__ __forceinline__ void store_tile(const MxGemmArgs &p, uint8_t *smem,
                                           const f32x4_t (&acc)[FM][FN], int m0, int n0, int mr,
                                           int nr, int wm0, int wn0, bool has) {
  constexpr int CLD = BN + 8, CPR = BN / 8;
  uint16_t *ct = reinterpret_cast<uint16_t *>(smem);
  const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  if (has) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const uint2 o = make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]),
                                   pack_bf16x2(acc[i][j][2], acc[i][j][3]));
        *reinterpret_cast<uint2 *>(ct + (wm0 + i * 16 + r) * CLD + wn0 + j * 16 + 4 * g) = o;
      }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < BM * CPR; c += NT) {
    const int row = c / CPR, col = (c - row * CPR) * 8;
    if (row >= mr || col >= nr) continue;
    const uint16_t *src = ct + row * CLD + col;
    uint16_t *dst = p.y + (int64_t)(m0 + row) * p.ldy + n0 + col;
    if (col + 8 <= nr) {
      const uint4 v = *reinterpret_cast<const uint4 *>(src);
      __builtin_memcpy(dst, &v, 16);  // any alignment
    } else {
      for (int e = 0; e < 8 && col + e < nr; ++e) dst[e] = src[e];
    }
  }
}

// BM rows of x by BN rows of W, k in tiles of KS steps of four blocks (128
// elements), ST tiles in an LDS ring, WM x WN waves -- KG times as many with
// the steps of a tile shared out over KG groups, whose sums meet in LDS.
//
// LDS holds a tile's codes row by row, the 16-byte chunks of a row permuted
// so that the eight rows a 128-byte LDS cycle serves take different banks:
// chunk c of row r at c ^ (r & 7), in 64-byte rows at c ^ (r / 2 & 3).
// Scales: 16 bytes a row, for four steps at a time, in a ring of their own.
//
// Few rows: bound by W's bytes (1 x 9216 x 8192 fp8 7 us of kernel, 40 MB) or,
// where those are few, by the latency of a step (256 x 4096 x 4096 fp8, one
// 64 x 64 tile a CU: 8.5 us of kernel, 0.23 a step).
template <int BM, int BN, int WM, int WN, int KG, int KS, int ST, int XF>
struct Tile {
  static constexpr int NW = WM * WN * KG, NT = 64 * NW;
  static constexpr int XB = (XF == kFp8 ? 128 : 64) * KS;  // bytes a row and tile
  static constexpr int WB = 64 * KS;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int X_BYTES = BM * XB, W_BYTES = BN * WB, STAGE = X_BYTES + W_BYTES;
  static constexpr int GT = 4 / KS;                       // tiles a group of scales serves
  // groups in the ring: those of the ST tiles in it, and the one being read
  static constexpr int SR = GT == 1 ? ST : (ST - 1 + GT - 1) / GT + 1;
  static constexpr int BMS = (BM + 63) / 64 * 64, BNS = (BN + 63) / 64 * 64;  // rows of scales loaded
  static constexpr int S_BYTES = (BMS + BNS) * 16;
  // instructions a wave issues a tile (1 KiB of codes or 64 rows of scales
  // each); where there are fewer than waves, several load the same
  static constexpr int XI = X_BYTES / 1024, WI = W_BYTES / 1024, SI = (BMS + BNS) / 64;
  static constexpr int XL = (XI + NW - 1) / NW, WL = (WI + NW - 1) / NW, SL = (SI + NW - 1) / NW;
  // waits count the codes' loads only: a group of scales goes ahead of its
  // first tile's codes, so it has landed when they have
  static constexpr int LOADS = XL + WL + (GT == 1 ? SL : 0);
  static constexpr int CLD = BN + 8;
  static constexpr int RING = ST * STAGE + SR * S_BYTES;
  static constexpr int EPI = std::max(BM * CLD * 2, (KG - 1) * BM * BN * 4);
  static constexpr int SMEM = std::max(RING, EPI);
  static_assert(KS % KG == 0, "steps to share");
  static_assert(KS == 1 || KS == 2 || KS == 4, "steps");
  static_assert(X_BYTES % 1024 == 0 && W_BYTES % 1024 == 0, "whole instructions");
  static_assert(FM * WM * 16 == BM && FN * WN * 16 == BN, "tile split");
  static_assert((ST - 1) * LOADS < 64, "vmcnt");
};

// LDS place of 16-byte chunk c in a row of RB bytes.
template <int RB>
__device__ __forceinline__ int place(int row, int c) {
  return row * RB + ((RB == 64 ? c ^ ((row >> 1) & 3) : c ^ (row & 7)) * 16);
}

template <int BM, int BN, int WM, int WN, int KG, int KS, int ST, int XF>
__global__ __launch_bounds__(64 * WM * WN * KG) void k_gemm_mx_tile(MxGemmArgs p) {
  using T = Tile<BM, BN, WM, WN, KG, KS, ST, XF>;
  static_assert(T::SMEM <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::SMEM];
  int tm, tn;
  tile_of(p, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int mr = min(BM, p.M - m0), nr = min(BN, p.N - n0);
  const Sources src = sources<XF>(p, m0, n0, mr, nr);
  const i32x4_t rx = src.x, rw = src.w, rxs = src.xs, rws = src.ws;
  const int nk = (p.nb + 4 * KS - 1) / (4 * KS);
  const uint32_t base = lds_addr(smem);

  // this lane's source offsets, and the block of the tile each one is in
  uint32_t vx[T::XL], vw[T::WL], vs[T::SL], bx[T::XL], bw[T::WL];
#pragma unroll
  for (int i = 0; i < T::XL; ++i) {
    const int at = (wave * T::XL + i) % T::XI * 64 + lane, row = at / (T::XB / 16);
    const int c = (place<T::XB>(row, at % (T::XB / 16)) - row * T::XB) >> 4;
    vx[i] = (uint32_t)(row * p.ldx + c * 16);
    bx[i] = XF == kFp8 ? c >> 1 : c;
  }
#pragma unroll
  for (int i = 0; i < T::WL; ++i) {
    const int at = (wave * T::WL + i) % T::WI * 64 + lane, row = at / (T::WB / 16);
    const int c = (place<T::WB>(row, at % (T::WB / 16)) - row * T::WB) >> 4;
    vw[i] = (uint32_t)(row * p.ldw + c * 16);
    bw[i] = c;
  }
#pragma unroll
  for (int i = 0; i < T::SL; ++i) {
    const int ins = (wave * T::SL + i) % T::SI, row = ins * 64 + lane;  // x's rows, then W's
    vs[i] = ins < T::BMS / 64 ? (uint32_t)(row * p.ldxs) : (uint32_t)((row - T::BMS) * p.ldws);
  }
  // The scales of the group that starts with tile kt, if one does; they are
  // issued ahead of the tile's codes, so they have landed when those have.
  auto issue_scales = [&](int kt) {
    if (T::GT > 1 && kt % T::GT != 0) return;
    const int grp = kt / T::GT;
    const uint32_t to = base + ST * T::STAGE + (uint32_t)(grp % T::SR) * T::S_BYTES;
#pragma unroll
    for (int i = 0; i < T::SL; ++i) {
      const int ins = (wave * T::SL + i) % T::SI;
      // a row's last group may take bytes of the next row, which no live
      // block uses, and past the last row nothing
      dma(ins < T::BMS / 64 ? rxs : rws, to + ins * 1024, vs[i], (uint32_t)grp * 16);
    }
  };
  // Load d of tile kt's codes: x's, then W's.  Blocks past the row's end and
  // tiles past the last load nothing (zeros), so the count of loads never
  // changes.
  constexpr int kLoads = T::XL + T::WL;
  auto issue_codes = [&](int d, int kt, uint32_t stage) {
    const int left = p.nb - 4 * KS * kt;  // blocks from this tile on
    const uint32_t to = base + stage * T::STAGE;
    if (d < T::XL) {
      const int i = d;
      dma(rx, to + (wave * T::XL + i) % T::XI * 1024, (int)bx[i] < left ? vx[i] : kOob,
          (uint32_t)kt * T::XB);
    } else {
      const int i = d - T::XL;
      dma(rw, to + T::X_BYTES + (wave * T::WL + i) % T::WI * 1024, (int)bw[i] < left ? vw[i] : kOob,
          (uint32_t)kt * T::WB);
    }
  };
  auto issue = [&](int kt, uint32_t stage) {
    issue_scales(kt);
#pragma unroll
    for (int d = 0; d < kLoads; ++d) issue_codes(d, kt, stage);
  };

  f32x4_t acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int kg = KG == 1 ? 0 : wave / (WM * WN), wt = KG == 1 ? wave : wave % (WM * WN);
  const int wm0 = (wt / WN) * (T::FM * 16), wn0 = (wt % WN) * (T::FN * 16);

  // Operands of step s of tile kt.  The scale of a block past the row's end
  // is that of a block inside it: it meets zero codes, and is NaN only where
  // the row is.
  auto scale_at = [&](int kt, int s) {
    const int blk = (kt % T::GT * KS + s) * 4 + g;
    return (kt / T::GT % T::SR) * T::S_BYTES + (4 * (kt * KS + s) + g < p.nb ? blk : 0);
  };
  // A lane's rows are 16 apart, so one address and immediate offsets reach
  // all of a step's fragments.
  auto w_at = [&](uint32_t stage, int s) {
    return smem + stage * T::STAGE + T::X_BYTES + wn0 * T::WB + place<T::WB>(r, 4 * s + g);
  };
  auto x_at = [&](uint32_t stage, int s, int half) {  // half: of an fp8 fragment
    return smem + stage * T::STAGE + wm0 * T::XB +
           place<T::XB>(r, XF == kFp8 ? 8 * s + 4 * half + g : 4 * s + g);
  };
  const uint8_t *sw_at = smem + ST * T::STAGE + (T::BMS + wn0 + r) * 16;
  const uint8_t *sx_at = smem + ST * T::STAGE + (wm0 + r) * 16;
  auto read_w = [&](const uint8_t *at, int sc_at, int j, i32x4_t &f, uint32_t &sc) {
    f = *reinterpret_cast<const i32x4_t *>(at + j * 16 * T::WB);
    sc = (sw_at + sc_at)[j * 256];
  };
  auto read_x = [&](const uint8_t *at, const uint8_t *at2, int sc_at, int i, frag_t<XF> &f, uint32_t &sc) {
    if constexpr (XF == kFp8)
      f = frag8(*reinterpret_cast<const i32x4_t *>(at + i * 16 * T::XB),
                *reinterpret_cast<const i32x4_t *>(at2 + i * 16 * T::XB));
    else
      f = *reinterpret_cast<const i32x4_t *>(at + i * 16 * T::XB);
    sc = (sx_at + sc_at)[i * 256];
  };
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) issue(s, s);
  uint32_t stage = 0, next = ST - 1;
  for (int kt = 0; kt < nk; ++kt) {
    wait_vm<(ST - 2) * T::LOADS>();  // tile kt has landed
    barrier();                       // every wave's part has, and tile kt - 1 is free
    issue(kt + ST - 1, next);
    next = next + 1 == ST ? 0 : next + 1;
#pragma unroll
    for (int u = 0; u < KS / KG; ++u) {
      const int s = kg + KG * u, sc = scale_at(kt, s);
      const uint8_t *wa = w_at(stage, s), *xa = x_at(stage, s, 0), *xb = x_at(stage, s, 1);
      i32x4_t wf[T::FN];
      uint32_t swb[T::FN];
#pragma unroll
      for (int j = 0; j < T::FN; ++j) read_w(wa, sc, j, wf[j], swb[j]);
#pragma unroll
      for (int i = 0; i < T::FM; ++i) {
        frag_t<XF> xf;
        uint32_t sxb;
        read_x(xa, xb, sc, i, xf, sxb);
#pragma unroll
        for (int j = 0; j < T::FN; ++j) acc[i][j] = mfma<XF>(wf[j], xf, acc[i][j], swb[j], sxb);
      }
    }
    stage = stage + 1 == ST ? 0 : stage + 1;
  }
  wait_vm<0>();

  if constexpr (KG > 1) {  // the groups' sums, in the groups' order
    __syncthreads();
    f32x4_t *part = reinterpret_cast<f32x4_t *>(smem);
    auto at = [&](int q, int i, int j) {
      return (((q - 1) * WM * WN + wt) * T::FM * T::FN + i * T::FN + j) * 64 + lane;
    };
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) part[at(kg, i, j)] = acc[i][j];
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
          for (int q = 1; q < KG; ++q) acc[i][j] += part[at(q, i, j)];
    }
  }

  __syncthreads();
  store_tile<BM, BN, T::FM, T::FN, T::NT>(p, smem, acc, m0, n0, mr, nr, wm0, wn0, kg == 0);
}

// ---------------------------------------------------------------------------
// Large tiles: every load a run of 128 bytes of a row, and so W's pairs of
// steps also where x goes by steps: a load into LDS costs a CU 2.2 cycles a
// 128-byte line (measured; half a line costs as much).  At 8192 x 9216 x 8192
// fp4 that is 90 of the 280 us that the loads alone take; the rest is their
// wait for the L2s' answers, with one pair of tiles on its way (10 TB/s).
// ---------------------------------------------------------------------------

// k runs in pairs of steps (256 elements).  W's ring holds two pairs, x's STX
// tiles of 128 bytes a row: a pair in fp4, a step in fp8; scales SGB bytes a
// row (SGB / 8 pairs), two groups.
// 8192 x 9216 x 8192: fp4 340 us (3.6 PFLOP/s; a loop of the products on
// registers reaches 7.1), fp8 466 (2.7; 4.8); 512 x 9216 x 8192 fp8 43 us
// (three sets of inputs or more in turn; with one, 310, 450 and 39).
// Without the loads into LDS they take 268, 400 and 32, the loads alone 280,
// 310 and 29: bound by neither alone, but by how far the two overlap.
template <int BM, int BN, int WM, int WN, int STX, int SGB, int XF>
struct Big {
  static constexpr int NW = WM * WN;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int X_STAGE = BM * 128, W_STAGE = BN * 128;
  static constexpr int BNS = (BN + 63) / 64 * 64;
  static constexpr int S_STAGE = (BM + BNS) * SGB;
  static constexpr int W0 = STX * X_STAGE, S0 = W0 + 2 * W_STAGE;
  static constexpr int XL = X_STAGE / 1024 / NW, WI = W_STAGE / 1024, WL = (WI + NW - 1) / NW;
  static constexpr int SRI = 16384 / SGB / 16;  // rows of scales to an instruction
  static constexpr int SI = (BM + BNS) / SRI, SL = (SI + NW - 1) / NW;
  static constexpr int GP = SGB / 8;            // pairs to a group of scales
  static constexpr int CLD = BN + 8;
  static constexpr int SMEM = std::max(S0 + 2 * S_STAGE, BM * CLD * 2);
  static_assert(X_STAGE % (1024 * NW) == 0, "whole instructions");
  static_assert(FM * WM * 16 == BM && FN * WN * 16 == BN && FM % 2 == 0, "tile split");
  static_assert(BM % 64 == 0 && W_STAGE % 1024 == 0 && (SGB == 16 || SGB == 32), "whole instructions");
};

template <int BM, int BN, int WM, int WN, int STX, int SGB, int XF>
__global__ __launch_bounds__(64 * WM * WN) void k_gemm_mx_big(MxGemmArgs p) {
  using T = Big<BM, BN, WM, WN, STX, SGB, XF>;
  static_assert(XF == kFp8 || STX == 2, "fp4: the tiles of x and W of a pair go together");
  static_assert(T::SMEM <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::SMEM];
  int tm, tn;
  tile_of(p, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mr = min(BM, p.M - m0), nr = min(BN, p.N - n0);
  const Sources src = sources<XF>(p, m0, n0, mr, nr);
  const i32x4_t rx = src.x, rw = src.w, rxs = src.xs, rws = src.ws;
  const uint32_t ldx = (uint32_t)p.ldx, ldw = (uint32_t)p.ldw;
  const uint32_t ldxs = (uint32_t)p.ldxs, ldws = (uint32_t)p.ldws;
  const int np = (p.nb + 7) >> 3;
  const uint32_t base = lds_addr(smem);

  // Sources.  A code instruction takes eight rows' 128 bytes, lane l chunk
  // (l & 7) ^ (l / 8) of row l / 8, which is its place in LDS (place<128>).
  // A scale instruction takes SRI rows; with 32 bytes a row the halves of
  // rows 4 .. 7 of eight change places, for the banks.
  const int c = (lane & 7) ^ (lane >> 3);
  const uint32_t vx = (lane >> 3) * ldx + c * 16, vw = (lane >> 3) * ldw + c * 16;
  auto issue_scales = [&](int pair) {  // of the group that starts with this pair, if one does
    if (pair % T::GP != 0) return;
    const int srow = SGB == 16 ? lane : lane >> 1;
    const int sseg = SGB == 16 ? 0 : ((lane & 1) ^ ((srow >> 2) & 1)) * 16;
    const uint32_t grp = (uint32_t)pair / T::GP;
    const uint32_t to = base + T::S0 + (grp & 1) * T::S_STAGE;
#pragma unroll
    for (int i = 0; i < T::SL; ++i) {
      const int ins = (wave * T::SL + i) % T::SI, row = ins * T::SRI;
      if (row < BM) dma(rxs, to + ins * 1024, srow * ldxs + sseg, row * ldxs + grp * SGB);
      else dma(rws, to + ins * 1024, srow * ldws + sseg, (row - BM) * ldws + grp * SGB);
    }
  };
  // tile t of x (a pair in fp4, a step in fp8), tile t of W (a pair); blocks
  // past the row's end load nothing (zeros), so the count of loads is fixed
  auto load_x = [&](int i, int t, uint32_t stage) {
    const int ins = wave * T::XL + i;
    const bool live = XF == kFp8 ? 4 * t + (c >> 1) < p.nb : 8 * t + c < p.nb;
    dma(rx, base + stage * T::X_STAGE + ins * 1024, live ? vx : kOob, ins * 8 * ldx + (uint32_t)t * 128);
  };
  auto load_w = [&](int i, int t) {
    const int ins = (wave * T::WL + i) % T::WI;
    dma(rw, base + T::W0 + (t & 1) * T::W_STAGE + ins * 1024, 8 * t + c < p.nb ? vw : kOob,
        ins * 8 * ldw + (uint32_t)t * 128);
  };

  f32x4_t acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int wm0 = (wave / WN) * (T::FM * 16), wn0 = (wave % WN) * (T::FN * 16);

  // One step's operands in registers; each fragment's next value is read as
  // soon as its last product is issued.
  constexpr int H = T::FM / 2, RX = T::FN > 2 ? T::FN - 2 : 1;
  i32x4_t wf[T::FN];
  frag_t<XF> xf[T::FM];
  uint32_t swb[T::FN], sxb[T::FM];
  // scale byte offset of this lane's block of step s (0, 1) of a pair; of a
  // block past the row's end: of the group's first (it meets zero codes, and
  // is NaN only where the row is)
  auto scale_at = [&](int pair, int s) {
    const int g = lane >> 4;
    const int b = 8 * pair + 4 * s + g < p.nb ? (pair % T::GP * 2 + s) * 4 + g : 0;
    return T::S0 + ((pair / T::GP) & 1) * T::S_STAGE + (lane & 15) * SGB +
           (SGB == 16 ? b : b ^ ((lane & 4) << 2));
  };
  // fragment i of x for step s of a pair, stage its place in the ring
  auto read_x = [&](int i, int pair, int s, uint32_t stage) {
    const int g = lane >> 4;
    const uint8_t *sx = smem + stage * T::X_STAGE + wm0 * 128 + i * 2048;
    if constexpr (XF == kFp8)
      xf[i] = frag8(*reinterpret_cast<const i32x4_t *>(sx + place<128>(lane & 15, g)),
                    *reinterpret_cast<const i32x4_t *>(sx + place<128>(lane & 15, g + 4)));
    else
      xf[i] = *reinterpret_cast<const i32x4_t *>(sx + place<128>(lane & 15, 4 * s + g));
    sxb[i] = smem[scale_at(pair, s) + (wm0 + i * 16) * SGB];
  };
  auto read_w = [&](int j, int pair, int s) {
    wf[j] = *reinterpret_cast<const i32x4_t *>(smem + T::W0 + (pair & 1) * T::W_STAGE + (wn0 + j * 16) * 128 +
                                               place<128>(lane & 15, 4 * s + (lane >> 4)));
    swb[j] = smem[scale_at(pair, s) + (BM + wn0 + j * 16) * SGB];
  };
  auto next_stage = [](uint32_t s) { return s + 1 == STX ? 0u : s + 1; };

  // prologue: pair 0 in, pair 1 (and, in fp8, half of it) on the way
  issue_scales(0);
  issue_scales(1);
#pragma unroll
  for (int i = 0; i < T::WL; ++i) load_w(i, 0);
#pragma unroll
  for (int t = 0; t < STX; ++t)
#pragma unroll
    for (int i = 0; i < T::XL; ++i) load_x(i, t, t);
#pragma unroll
  for (int i = 0; i < T::WL; ++i) load_w(i, 1);
  wait_vm<(STX - 1) * T::XL + T::WL>();
  barrier();
  uint32_t stage = 0;  // of x's current tile
#pragma unroll
  for (int i = 0; i < H; ++i) read_x(i, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < T::FN; ++j) read_w(j, 0, 0);

  for (int pr = 0; pr < np; ++pr) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      // the upper rows' products, the lower rows of x read meanwhile
#pragma unroll
      for (int j = 0; j < T::FN; ++j) {
        // (all of them ahead of the last products, which cover their way)
#pragma unroll
        for (int i = H * j / RX; i < (j < RX ? H * (j + 1) / RX : 0); ++i) read_x(H + i, pr, s, stage);
#pragma unroll
        for (int i = 0; i < H; ++i) acc[i][j] = mfma<XF>(wf[j], xf[i], acc[i][j], swb[j], sxb[i]);
        __builtin_amdgcn_sched_barrier(0);
      }
      // every wave has read the tile of x (with s = 1, and of W), and the
      // next one has landed: in fp8 the tiles of x after it, and with s = 0
      // the next of W, may be on the way
      if (XF == kFp8 || s == 1) {
        if (XF != kFp8) wait_vm<0>();
        else if (s == 0) wait_vm<(STX - 2) * T::XL + T::WL>();
        else wait_vm<(STX - 2) * T::XL>();
        barrier();
        if (s == 1) issue_scales(pr + 2);
      }
      // the lower rows' products, the next step's upper rows of x and, column
      // by column, W read and the freed tiles refilled meanwhile; past the
      // last pair zeros are read and not used
      const int prn = s == 1 ? pr + 1 : pr, sn = s ^ 1;
      const uint32_t freed = stage;
      if (XF == kFp8 || s == 1) stage = next_stage(stage);
      __builtin_amdgcn_sched_barrier(0);
      const int nx = XF == kFp8 || s == 1 ? T::XL : 0, nl = nx + (s == 1 ? T::WL : 0);
#pragma unroll
      for (int j = 0; j < T::FN; ++j) {
#pragma unroll
        for (int i = H; i < T::FM; ++i) acc[i][j] = mfma<XF>(wf[j], xf[i], acc[i][j], swb[j], sxb[i]);
        read_w(j, prn, sn);
#pragma unroll
        for (int i = H * j / RX; i < (j < RX ? H * (j + 1) / RX : 0); ++i) read_x(i, prn, sn, stage);
#pragma unroll
        for (int d = nl * j / T::FN; d < nl * (j + 1) / T::FN; ++d) {
          if (d < nx) load_x(d, XF == kFp8 ? 2 * pr + s + STX : pr + 2, freed);
          else load_w(d - nx, pr + 2);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // the sums stay where they are (left to itself the compiler gives the
      // two steps of the loop different registers for them and spills)
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) {
          if constexpr (T::NW == 4) asm volatile("" : "+a"(acc[i][j]));
          else asm volatile("" : "+v"(acc[i][j]));
        }
    }
  }
  wait_vm<0>();  // the loads past the end have landed: LDS is free
  __syncthreads();
  store_tile<BM, BN, T::FM, T::FN, 64 * T::NW>(p, smem, acc, m0, n0, mr, nr, wm0, wn0, true);
}

template <int BM, int BN, int WM, int WN, int STX, int SGB, int XF>
void launch_big(MxGemmArgs a, hipStream_t st) {
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + BN - 1) / BN;
  hipLaunchKernelGGL((k_gemm_mx_big<BM, BN, WM, WN, STX, SGB, XF>), dim3((unsigned)(a.tiles_m * a.tiles_n)),
                     dim3(64 * WM * WN), 0, st, a);
}

template <int BM, int BN, int WM, int WN, int KG, int KS, int ST, int XF>
void launch_tile(MxGemmArgs a, hipStream_t st) {
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + BN - 1) / BN;
  hipLaunchKernelGGL((k_gemm_mx_tile<BM, BN, WM, WN, KG, KS, ST, XF>),
                     dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(64 * WM * WN * KG), 0, st, a);
}

// The tile shape.  With t tiles over the 256 CUs, of which a CU holds `fit` at
// once, and steps of 128 elements, a shape's time is taken as
//   s + ceil(t / 256 fit) (e + c steps) + (ceil(t / 256) w + t / 256 f) steps
// in us: what a round of workgroups takes alone, what those that share a CU
// and those on other CUs add.  The five numbers are least-squares fits (none
// negative) of each shape's times at up to 160 sizes per format (20 values of
// M from 1 to 8192, d x k of 9216 x 8192, 4096 x 4096, 5120 x 5120, 2048 x
// 4096, 1024 x 1024, 1024 x 8192, 9216 x 512 and 8192 x 1024), good to 2 - 8%;
// the choice is within 1% of the best of 37 shapes tried, on the mean.  Of
// those the table holds the ones without which that gets worse: by the model,
// leaving one out costs 0.06 to 4% on the mean of the fitted sizes (fp4's 64 x
// 96 tiles 0.006%, its large 64 x 128 ones nothing there) and 0.02 to 6% over
// M from 1 to 8192, k and d from 64 to 8192 and 9216, uniform in the logarithm.
// Over those the least used are fp4's 192 x 128 tiles (4 of 20000 sizes,
// 0.002%; 0.06% of the fitted ones) and fp8's 32 x 80 (13, 0.006%; 0.08%).
// 128 x 9216 x 8192 fp8 takes 20.1 us (64 x 128 tiles 25), 256 x 9216 x 8192
// 28.6 (128 x 144 tiles 41), 512 x 5120 x 5120 20.3 (28).
struct Shape {
  int bm, bn, fit;
  int ring;  // elements of k that the longest LDS ring holds
  float s, e, c, w, f;
  void (*launch)(MxGemmArgs, hipStream_t);
};
constexpr int fit(int smem, int waves) { return std::max(1, std::min(160 * 1024 / smem, 16 / waves)); }

template <int BM, int BN, int WM, int WN, int KG, int KS, int ST, int XF>
constexpr Shape tile(float s, float e, float c, float w, float f) {
  using T = Tile<BM, BN, WM, WN, KG, KS, ST, XF>;
  return {BM, BN, fit(T::SMEM, T::NW), 128 * KS * std::max(ST, T::SR * T::GT), s, e, c, w, f,
          launch_tile<BM, BN, WM, WN, KG, KS, ST, XF>};
}
template <int BM, int BN, int WM, int WN, int STX, int SGB, int XF>
constexpr Shape big(float s, float e, float c, float w, float f) {
  using T = Big<BM, BN, WM, WN, STX, SGB, XF>;
  return {BM, BN, fit(T::SMEM, T::NW), 2 * SGB * 32, s, e, c, w, f, launch_big<BM, BN, WM, WN, STX, SGB, XF>};
}

const Shape kShapes8[] = {
    tile<16, 16, 1, 1, 4, 4, 8, kFp8>(1.28f, 1.60f, 0.054f, 0.f, 0.006f),
    tile<16, 64, 1, 1, 4, 4, 4, kFp8>(1.18f, 1.82f, 0.086f, 0.f, 0.015f),
    tile<32, 48, 1, 1, 4, 4, 4, kFp8>(1.24f, 2.13f, 0.102f, 0.f, 0.016f),
    tile<32, 64, 1, 2, 4, 4, 4, kFp8>(1.10f, 2.08f, 0.112f, 0.f, 0.029f),
    tile<32, 80, 1, 1, 4, 4, 3, kFp8>(1.30f, 2.74f, 0.159f, 0.f, 0.018f),
    tile<48, 64, 1, 2, 4, 4, 3, kFp8>(1.21f, 2.25f, 0.149f, 0.f, 0.037f),
    tile<64, 64, 2, 2, 2, 2, 4, kFp8>(0.94f, 2.12f, 0.201f, 0.f, 0.037f),
    tile<64, 80, 2, 1, 2, 2, 4, kFp8>(0.87f, 2.90f, 0.227f, 0.f, 0.038f),
    big<64, 96, 2, 2, 3, 16, kFp8>(0.89f, 2.29f, 0.173f, 0.079f, 0.063f),
    big<64, 128, 2, 2, 3, 16, kFp8>(0.61f, 2.79f, 0.148f, 0.128f, 0.078f),
    big<128, 96, 4, 1, 2, 32, kFp8>(1.04f, 2.54f, 0.331f, 0.036f, 0.215f),
    big<128, 112, 4, 1, 3, 32, kFp8>(0.66f, 3.68f, 0.356f, 0.f, 0.102f),
    big<128, 144, 4, 1, 3, 32, kFp8>(0.73f, 4.24f, 0.409f, 0.f, 0.145f),
    big<256, 128, 4, 2, 3, 16, kFp8>(0.f, 4.64f, 0.591f, 0.f, 0.307f),
    big<256, 160, 4, 2, 3, 16, kFp8>(0.32f, 5.12f, 0.663f, 0.f, 0.351f),
    big<256, 192, 4, 2, 3, 16, kFp8>(0.f, 5.76f, 0.782f, 0.f, 0.398f),
    big<256, 256, 4, 2, 2, 16, kFp8>(0.09f, 6.24f, 1.034f, 0.f, 0.676f),
};
const Shape kShapes4[] = {
    tile<16, 16, 1, 1, 4, 4, 8, kFp4>(1.29f, 1.67f, 0.f, 0.035f, 0.001f),
    tile<16, 64, 1, 1, 4, 4, 4, kFp4>(1.22f, 1.68f, 0.078f, 0.f, 0.012f),
    tile<32, 32, 1, 1, 4, 4, 4, kFp4>(1.43f, 1.59f, 0.f, 0.060f, 0.004f),
    tile<32, 48, 1, 1, 4, 4, 4, kFp4>(1.19f, 1.94f, 0.077f, 0.f, 0.014f),
    tile<32, 64, 1, 2, 4, 4, 4, kFp4>(1.12f, 1.84f, 0.090f, 0.f, 0.028f),
    tile<64, 48, 2, 1, 2, 2, 4, kFp4>(1.20f, 1.99f, 0.049f, 0.084f, 0.013f),
    tile<64, 64, 2, 2, 2, 2, 4, kFp4>(1.02f, 1.99f, 0.007f, 0.134f, 0.027f),
    tile<64, 80, 2, 1, 2, 4, 2, kFp4>(0.71f, 3.00f, 0.078f, 0.086f, 0.034f),
    tile<64, 96, 2, 2, 2, 2, 4, kFp4>(0.85f, 2.40f, 0.181f, 0.f, 0.047f),
    tile<64, 128, 2, 2, 2, 2, 4, kFp4>(0.79f, 2.61f, 0.202f, 0.f, 0.071f),
    big<64, 128, 2, 2, 2, 16, kFp4>(0.53f, 2.71f, 0.186f, 0.041f, 0.105f),
    big<128, 64, 4, 1, 2, 32, kFp4>(0.51f, 2.82f, 0.196f, 0.020f, 0.103f),
    big<128, 96, 4, 1, 2, 32, kFp4>(0.75f, 3.11f, 0.196f, 0.074f, 0.098f),
    big<128, 128, 2, 2, 2, 16, kFp4>(0.17f, 4.01f, 0.169f, 0.137f, 0.121f),
    big<192, 128, 2, 2, 2, 16, kFp4>(0.49f, 4.17f, 0.363f, 0.f, 0.180f),
    big<256, 160, 4, 2, 2, 16, kFp4>(0.22f, 5.01f, 0.440f, 0.f, 0.281f),
    big<256, 192, 4, 2, 2, 16, kFp4>(0.f, 5.65f, 0.486f, 0.f, 0.312f),
    big<256, 256, 4, 2, 2, 16, kFp4>(0.f, 6.40f, 0.627f, 0.f, 0.448f),
};

template <size_t N>
const Shape &best_of(const Shape (&shapes)[N], const MxGemmArgs &a) {
  const Shape *best = nullptr;
  double least = 0;
  const double steps = (a.nb + 3) / 4;
  for (const Shape &h : shapes) {
    const int64_t tiles = ((int64_t)(a.M + h.bm - 1) / h.bm) * ((a.N + h.bn - 1) / h.bn);
    const double rounds = (double)((tiles + 256 * h.fit - 1) / (256 * h.fit)), cu = (double)((tiles + 255) / 256);
    const double t = h.s + rounds * (h.e + h.c * steps) + (cu * h.w + (double)tiles / 256 * h.f) * steps;
    if (best == nullptr || t < least) {
      best = &h;
      least = t;
    }
  }
  return *best;
}

// slabs whose grids stay far below what a launch takes
constexpr int64_t kSlab = int64_t(1) << 18;

}  // namespace

int gemm_mx_shape(int64_t M, int64_t k, int64_t d, int32_t xfmt, int32_t out[3]) {
  MxGemmArgs a{};
  a.M = (int32_t)std::min(kSlab, M);
  a.N = (int32_t)std::min(kSlab, d);
  a.nb = (int32_t)((k + kBlock - 1) / kBlock);
  const Shape &s = xfmt == kFp8 ? best_of(kShapes8, a) : best_of(kShapes4, a);
  out[0] = s.bm;
  out[1] = s.bn;
  out[2] = s.ring;
  return (int)(&s - (xfmt == kFp8 ? kShapes8 : kShapes4));
}

hipError_t launch_gemm_mx(const MxGemmArgs &all, hipStream_t st) {
  for (int64_t m0 = 0; m0 < all.M; m0 += kSlab)
    for (int64_t n0 = 0; n0 < all.N; n0 += kSlab) {
      MxGemmArgs a = all;
      a.M = (int32_t)std::min(kSlab, all.M - m0);
      a.N = (int32_t)std::min(kSlab, all.N - n0);
      a.x += m0 * a.ldx;
      a.xs += m0 * a.ldxs;
      a.w += n0 * a.ldw;
      a.wsc += n0 * a.ldws;
      a.y += m0 * a.ldy + n0;
      (a.xfmt == kFp8 ? best_of(kShapes8, a) : best_of(kShapes4, a)).launch(a, st);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace lora
