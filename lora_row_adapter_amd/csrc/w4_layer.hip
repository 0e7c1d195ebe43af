// w4_layer.hip -- the 4-bit layer for at most 32 rows (include/lora_w4.h): what
// goes ahead of the product that adds the adapters' part itself (w4.hip).
//
// With so few rows a plan has little to sort, and its launch, and the fork and
// join beside the product, cost more than the rest of the layer.  Here each
// workgroup finds by itself which rows it serves: up to four with one adapter, and of
// their t one slice's next few ranks.  Workgroup 0 checks the rows, as the plan does,
// and writes which adapter each is to get.
//
// What bounds it are the bytes of A at many adapters, and at few what a CU takes
// in: 64 bytes a clock where a wave's load is one run of memory, as here (each lane
// eight columns of one row of A), a quarter of that where it is 16 rows of 64 bytes,
// as matrix instructions would have it.  At two slices of 64 ranks x 8192: one row
// 4.6 us, 2.2 MB of A (4.4 with 8 ranks; 2.2 of them the launch and the rows' checks;
// 10.5 with matrix instructions and all of k to a workgroup); 16 rows of 12 adapters
// 9.1 us, 26 MB; of 8 adapters of 4 to 64 ranks 7.4 us, 8.5 MB.
#include <algorithm>

#include "kernels.hpp"

namespace lora {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kRows = 4;    // of an adapter at a time
constexpr int kFill = 512;  // workgroups aimed at

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
  if (lane < a.M) {
    a.row[lane] = paged ? id : -1;
    for (int q = 0; q < a.n_slices; ++q) a.rank[q * a.M + lane] = paged ? a.sl[q].ranks[id] : 0;
  }
  const bool live = lane < a.M;
  const uint64_t ids = __ballot(live && id != -1 && !known), ranks = __ballot(live && known && !ranked),
                 pages = __ballot(live && ranked && !paged);
  if (lane == 0) {
    a.hdr[kHdrBadIds] = (int)__popcll(ids);
    a.hdr[kHdrBadRanks] = (int)__popcll(ranks);
    a.hdr[kHdrBadPages] = (int)__popcll(pages);
  }
}

// A_s[j][k .. k + 7]; zeros where its page is none of the pool's, as such a row's
// t is not used.
__device__ __forceinline__ u32x4_t load_a(const AdapterRef &ar, int64_t n_pages, int s, int j, int64_t k) {
  const int64_t off = ((int64_t)j * ar.k + k) * 2;
  const uint8_t *at = ar.A + (int64_t)s * ar.max_rank * ar.k * 2 + off;
  if (ar.pooled) {
    const int32_t pg = ar.page_table[(int64_t)s * ar.max_pages + (off >> ar.page_shift)];
    if (pg < 0 || pg >= n_pages) return u32x4_t{0, 0, 0, 0};
    at = ar.pool + ((int64_t)pg << ar.page_shift) + (off & (ar.page_bytes - 1));
  }
  return *reinterpret_cast<const u32x4_t *>(at);
}

template <int kCtrl>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), kCtrl, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// The sum over a wave's lanes.
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0xB1>(v);   // lanes 1 0 3 2
  v = add_dpp<0x4E>(v);   // lanes 2 3 0 1
  v = add_dpp<0x141>(v);  // lanes 7 .. 0
  v = add_dpp<0x140>(v);  // lanes 15 .. 0
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
__device__ __forceinline__ float bf16_at(u32x4_t v, int i) {
  return __builtin_bit_cast(float, i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
}

// kRanks: of a workgroup.
template <int kRanks>
__global__ __launch_bounds__(kThreads) void k_w4_shrink(W4Lora a, int jblocks) {
  __shared__ float part[kWaves][kRows * kRanks];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  touch(a);
  const int id = lane < a.M ? a.ids[lane] : -1;
  if (blockIdx.x == 0) {
    check_rows(a, id);
    return;
  }
  // the v-th group of kRows rows with one adapter: its first row, slice, ranks
  int b = blockIdx.x - 1;
  const int j0 = b % jblocks * kRanks;
  b /= jblocks;
  const int q = b % a.n_slices, v = b / a.n_slices;
  int same = 0;  // rows above this lane's with its adapter
  for (int i = 0; i + 1 < a.M; ++i) same += i < lane && __builtin_amdgcn_readlane(id, i) == id;
  const bool leads = id >= 0 && id < a.S && same % kRows == 0;
  const uint64_t all = __ballot(leads);
  const uint64_t found = __ballot(leads && (int)__popcll(all & ((uint64_t(1) << lane) - 1)) == v);
  if (found == 0) return;
  const int u = __builtin_ctzll(found);
  const int s = __builtin_amdgcn_readlane(id, u), from = __builtin_amdgcn_readlane(same, u);
  uint64_t mine = __ballot(id == s && same >= from && same < from + kRows);
  const SliceRef &sl = a.sl[q];
  const int rank = sl.ranks[s];
  const float scale = sl.scales[s];
  if (rank < 0 || rank > sl.ar.max_rank || pages_of(a, q, rank) < 0) return;
  const int n = (int)__popcll(mine);
  int row[kRows];
  const uint16_t *x[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    row[i] = mine != 0 ? __builtin_ctzll(mine) : row[i - 1];
    mine &= mine - 1;
    x[i] = a.x + (int64_t)row[i] * a.ldx;
  }
  float acc[kRows][kRanks] = {};
  if (j0 < rank) {
#pragma unroll 2
    for (int64_t k = threadIdx.x * 8; k < a.k; k += kThreads * 8) {
      u32x4_t av[kRanks], xv[kRows];
#pragma unroll
      for (int e = 0; e < kRanks; ++e)  // past the rank: the last again, not kept
        av[e] = load_a(sl.ar, a.n_pages[q], s, min(j0 + e, rank - 1), k);
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (i < n) xv[i] = *reinterpret_cast<const u32x4_t *>(x[i] + k);
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (i < n)
#pragma unroll
          for (int e = 0; e < kRanks; ++e)
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[i][e] = __builtin_fmaf(bf16_at(xv[i], c), bf16_at(av[e], c), acc[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (i < n)
#pragma unroll
      for (int e = 0; e < kRanks; ++e) {
        const float v = wave_sum(acc[i][e]);
        if (lane == 0) part[wave][i * kRanks + e] = v;
      }
  __syncthreads();
  if ((int)threadIdx.x < n * kRanks) {
    const int j = j0 + threadIdx.x % kRanks;
    float v = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += part[w][threadIdx.x];
    const float t = j < rank ? v * scale : 0.f;
    const uint16_t hi = f32_to_bf16_bits(t);
    const float rest = t - bf16_bits_to_f32(hi);
    int to = row[0];
#pragma unroll
    for (int i = 1; i < kRows; ++i) to = (int)threadIdx.x / kRanks == i ? row[i] : to;
    const int64_t o = ((int64_t)q * a.M + to) * a.Rp + j;
    if (j < a.Rp) {
      a.t_hi[o] = hi;
      a.t_lo[o] = rest - rest == 0.f ? f32_to_bf16_bits(rest) : 0;  // of an infinity or a NaN: nothing
    }
  }
}

}  // namespace

bool w4_lora_place(W4Lora &a, uint8_t *at, size_t bytes) {
  const size_t t = (size_t)a.n_slices * a.M * a.Rp * sizeof(uint16_t), rows = (size_t)a.M * sizeof(int32_t);
  a.t_hi = reinterpret_cast<uint16_t *>(at);
  a.t_lo = reinterpret_cast<uint16_t *>(at + t);
  a.row = reinterpret_cast<int32_t *>(at + 2 * t);
  a.rank = a.row + a.M;
  return 2 * t + rows * (1 + a.n_slices) <= bytes;
}

// At most, of kRows rows with one adapter.
static int groups_of(const W4Lora &a) { return std::min(a.M, std::min(a.M, a.S) + a.M / kRows); }

template <int kRanks>
static void launch_shrink(const W4Lora &a, hipStream_t st) {
  const int jblocks = (a.Rp + kRanks - 1) / kRanks;
  hipLaunchKernelGGL(k_w4_shrink<kRanks>, dim3((unsigned)(1 + groups_of(a) * a.n_slices * jblocks)), dim3(kThreads), 0, st, a,
                     jblocks);
}

hipError_t launch_w4_shrink(const W4Lora &a, hipStream_t st) {
  // as many ranks to a workgroup, up to four, as leave two workgroups for each CU where
  // the groups are as many as they can be
  const int64_t ranks = (int64_t)groups_of(a) * a.n_slices * a.Rp;
  if (ranks < 2 * kFill) launch_shrink<1>(a, st);
  else if (ranks < 4 * kFill) launch_shrink<2>(a, st);
  else launch_shrink<4>(a, st);
  return hipGetLastError();
}

}  // namespace lora
