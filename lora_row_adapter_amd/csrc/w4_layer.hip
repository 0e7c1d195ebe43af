// w4_layer.hip -- the 4-bit layer for at most 64 rows (include/lora_w4.h): what
// goes ahead of the product that adds the adapters' part itself (w4.hip).
//
// With so few rows a plan has little to sort and its launch, and the fork and
// join beside the product, cost more than the rest of the layer.  Here each
// workgroup finds by itself whether it has work: workgroup (row u, slice,
// sixteen ranks) serves all rows of row u's adapter unless an earlier row has the
// same one, and takes its sixteen rows of A over all of k (sixteen waves, every
// second kilobyte of it on its way at once).  Workgroup 0 checks the rows, as the plan
// does, and writes which adapter each is to get.
#include "kernels.hpp"

namespace lora {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

// Pages that adapter s needs in slice q (0 in slots), or -1: past its table.
__device__ __forceinline__ int64_t pages_of(const W4Lora &a, int q, int r) {
  const AdapterRef &ar = a.sl[q].ar;
  if (!ar.pooled) return 0;
  const int64_t n = ((int64_t)r * (ar.k + ar.d) * ar.elem_bytes + ar.page_bytes - 1) >> ar.page_shift;
  return n > ar.max_pages ? -1 : n;
}
__device__ __forceinline__ bool bad_page(const W4Lora &a, int q, int s, int64_t j) {
  const AdapterRef &ar = a.sl[q].ar;
  const int32_t pg = ar.page_table[(int64_t)s * ar.max_pages + j];
  return pg < 0 || (int64_t)pg >= a.n_pages[q];
}
__device__ __forceinline__ bool ranks_ok(const W4Lora &a, int s) {
  bool ok = true;
  for (int q = 0; q < a.n_slices; ++q) {
    const int r = a.sl[q].ranks[s];
    ok = ok && r >= 0 && r <= a.sl[q].ar.max_rank;
  }
  return ok;
}

// Each row's adapter, the counts of rows that name none they can have.
__device__ __forceinline__ void check_rows(const W4Lora &a, int id) {
  __shared__ uint32_t bad[kW4Rows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (threadIdx.x < kW4Rows) bad[threadIdx.x] = 0;
  __syncthreads();
  const bool known = id >= 0 && id < a.S;
  const bool ranked = known && ranks_ok(a, id);
  // this lane's row stands for its adapter: the first with it
  int lead = lane;
  uint64_t leads = 0;
  for (uint64_t left = __ballot(ranked); left != 0;) {
    const int f = __builtin_ctzll(left);
    const uint64_t mine = __ballot(ranked && id == __builtin_amdgcn_readlane(id, f));
    if (mine >> lane & 1) lead = f;
    leads |= uint64_t(1) << f;
    left &= ~mine;
  }
  // their pages, a wave for each (adapter, slice) in turn
  int e = 0;
  for (uint64_t left = leads; left != 0; left &= left - 1) {
    const int f = __builtin_ctzll(left);
    const int s = __builtin_amdgcn_readlane(id, f);
    for (int q = 0; q < a.n_slices; ++q, ++e) {
      if (e % kWaves != wave || !a.sl[q].ar.pooled) continue;
      const int64_t n = pages_of(a, q, a.sl[q].ranks[s]);
      bool b = n < 0;
#pragma unroll 4
      for (int64_t j = lane; j < n; j += 64) b |= bad_page(a, q, s, j);
      if (b) atomicOr(&bad[f], 1u);
    }
  }
  __syncthreads();
  if (wave != 0) return;
  const bool paged = ranked && bad[lead] == 0;
  if (lane < a.M) a.row[lane] = paged ? id : -1;
  const bool live = lane < a.M;
  const uint64_t ids = __ballot(live && id != -1 && !known), ranks = __ballot(live && known && !ranked),
                 pages = __ballot(live && ranked && !paged);
  if (lane == 0) {
    a.hdr[kHdrBadIds] = (int)__popcll(ids);
    a.hdr[kHdrBadRanks] = (int)__popcll(ranks);
    a.hdr[kHdrBadPages] = (int)__popcll(pages);
  }
}

__global__ __launch_bounds__(kThreads) void k_w4_shrink(W4Lora a, int jblocks) {
  __shared__ f32x4_t part[kWaves][64];
  __shared__ int rows[kW4Rows];
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int id = lane < a.M ? a.ids[lane] : -1;
  if (blockIdx.x == 0) {
    check_rows(a, id);
    return;
  }
  const int b = blockIdx.x - 1, u = b / (a.n_slices * jblocks), q = b / jblocks % a.n_slices, j0 = b % jblocks * 16;
  const int s = __builtin_amdgcn_readlane(id, u);
  if (s < 0 || s >= a.S) return;
  const uint64_t mine = __ballot(id == s);
  if (__builtin_ctzll(mine) != u) return;
  const SliceRef &sl = a.sl[q];
  const int rank = sl.ranks[s];
  if (j0 >= rank || !ranks_ok(a, s)) return;
  bool bad = false;
  for (int p = 0; p < a.n_slices; ++p) {
    const int64_t n = pages_of(a, p, a.sl[p].ranks[s]);
    bad |= n < 0;
    for (int64_t j = threadIdx.x; j < n; j += kThreads) bad |= bad_page(a, p, s, j);
  }
  const int cnt = (int)__popcll(mine);
  if (wave == 0 && (mine >> lane & 1)) rows[__popcll(mine & ((uint64_t(1) << lane) - 1))] = lane;
  if (__syncthreads_or(bad)) return;

  const float scale = sl.scales[s];
  for (int t0 = 0; t0 < cnt; t0 += 16) {
    const uint16_t *x = a.x + (int64_t)rows[min(t0 + r, cnt - 1)] * a.ldx;  // past the last: that, not kept
    const int j = min(j0 + r, rank - 1);                                      // likewise
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    constexpr int kSteps = 8;
    for (int64_t c = wave * (32 * kSteps); c < a.k; c += kWaves * 32 * kSteps) {
      u32x4_t xv[kSteps], av[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int64_t k = c + 32 * i + 8 * h;
        xv[i] = av[i] = u32x4_t{0, 0, 0, 0};
        if (k < a.k) {
          xv[i] = *reinterpret_cast<const u32x4_t *>(x + k);
          av[i] = *reinterpret_cast<const u32x4_t *>(adapter_a_ptr(sl.ar, s, rank, j, k));
        }
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xv[i]),
                                                      __builtin_bit_cast(bf16x8_t, av[i]), acc, 0, 0, 0);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      f32x4_t v = part[0][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += part[w][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (t0 + 4 * h + e >= cnt) continue;
        // zeros from the rank to the sixteen's end, where the product reads on
        const float t = j0 + r < rank ? v[e] * scale : 0.f;
        const uint16_t hi = f32_to_bf16_bits(t);
        const float rest = t - bf16_bits_to_f32(hi);
        const int64_t o = ((int64_t)q * a.M + rows[t0 + 4 * h + e]) * a.Rp + j0 + r;
        a.t_hi[o] = hi;
        // of an infinity or a NaN: nothing
        a.t_lo[o] = rest - rest == 0.f ? f32_to_bf16_bits(rest) : 0;
      }
    }
    __syncthreads();
  }
}

}  // namespace

size_t w4_lora_bytes(int64_t M, int32_t n_slices, int32_t R) {
  const int64_t Rp = (R + 31) & ~31;
  return (size_t)(n_slices * M * Rp * 4 + M * 4);
}

hipError_t launch_w4_shrink(const W4Lora &a, hipStream_t st) {
  int32_t R = 0;
  for (int q = 0; q < a.n_slices; ++q) R = R > a.sl[q].ar.max_rank ? R : a.sl[q].ar.max_rank;
  const int jblocks = (R + 15) / 16;
  hipLaunchKernelGGL(k_w4_shrink, dim3((unsigned)(1 + a.M * a.n_slices * jblocks)), dim3(kThreads), 0, st, a, jblocks);
  return hipGetLastError();
}

}  // namespace lora
