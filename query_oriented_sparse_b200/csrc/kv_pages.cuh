// A paged KV cache: pools of pages k / v [num_pages][h_kv][page_size][head_dim] and, per
// key and KV head, a record of accumulated attention weight [num_pages][h_kv][page_size]
// (fp32).  Position j of sequence b lies in page block_table[b][j / page_size], slot
// j % page_size.  This file holds the addressing and the two operators that move rows:
//
//   paged_append_kernel  new rows into the pages; a copy, bound by its bytes (or, for one
//                        token per sequence, by the launch).
//   evict_select_kernel  the rows to keep, per (sequence, KV head): the first `first` and
//                        the last `last` rows, and of the rest those with the most weight,
//                        ties to the lower position.  A radix select (cluster_select.cuh)
//                        over the rest of the sequence, ascending output without a sort.
//                        Bound by latency (staging, four passes, two walks): 30 us for 256
//                        rows of up to 16K keys, 22 us for 8 rows of 131072 over 16 CTAs each.
//   evict_copy_kernel    the kept rows and their records, in order, into other pages.
#pragma once
#include "cluster_select.cuh"
#include "tc_ptx.cuh"

namespace quoka {

// Where the K/V rows of (sequence, KV head, position) lie.  seq_len, block_table: paged
// (device memory); rows_per_head and a SeqTable: the contiguous cache.
struct KvView {
  const int32_t* seq_len;
  const int32_t* block_table;
  int max_pages, page_size, num_pages;
  int max_len;                     // the caller's bound on seq_len
  long long rows_per_head;
};

// Tokens of sequence b, held to [0, bound] (a length outside is reported).
__device__ __forceinline__ int paged_len(const int32_t* seq_len, int b, int bound) {
  const int n = __ldg(seq_len + b);
  if (n >= 0 && n <= bound) return n;
  flag_error(ERR_BAD_INDEX);
  return n < 0 ? 0 : bound;
}

// Page of position j of sequence b, or -1 (reported) when the table holds none there.
__device__ __forceinline__ int page_of(const KvView& kv, int b, int j, int* slot) {
  const int p = j / kv.page_size;
  *slot = j - p * kv.page_size;
  const int page = __ldg(kv.block_table + (size_t)b * kv.max_pages + p);
  if (page >= 0 && page < kv.num_pages) return page;
  flag_error(ERR_BAD_INDEX);
  return -1;
}

// Row (of head_dim elements) of position j in a pool; -1 when its page is bad.
__device__ __forceinline__ long long paged_row(const KvView& kv, int b, int g, int h_kv, int j) {
  int slot;
  const int page = page_of(kv, b, j, &slot);
  return page < 0 ? -1 : ((long long)page * h_kv + g) * kv.page_size + slot;
}

constexpr int PAGED_THREADS = 256;

// New rows k_new / v_new [batch][h_kv][n_new][D] of sequence b to positions start[b] + t,
// t < count[b] (all n_new when count is NULL).  One thread per 16-byte vector of a row.
// A row whose position has no page is reported and not written.
__global__ void __launch_bounds__(PAGED_THREADS)
paged_append_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, uint4* __restrict__ k,
                    uint4* __restrict__ v, float* __restrict__ record, const KvView kv,
                    const int32_t* __restrict__ start, const int32_t* __restrict__ count, int h_kv, int n_new,
                    int vpr, long long total) {
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (long long)gridDim.x * blockDim.x) {
    const long long row = e / vpr;
    const int vec = (int)(e - row * vpr);
    const long long bg = row / n_new;
    const int t = (int)(row - bg * n_new);
    const int b = (int)(bg / h_kv), g = (int)(bg - (long long)b * h_kv);
    if (count && t >= paged_len(count, b, n_new)) continue;
    const long long at = (long long)__ldg(start + b) + t;
    if (at < 0 || at >= (long long)kv.max_pages * kv.page_size) {
      flag_error(ERR_BAD_INDEX);
      continue;
    }
    const long long dst = paged_row(kv, b, g, h_kv, (int)at);
    if (dst < 0) continue;
    k[dst * vpr + vec] = __ldg(k_new + e);
    v[dst * vpr + vec] = __ldg(v_new + e);
    if (record && vec == 0) record[dst] = 0.f;
  }
}

// How many rows sequence b keeps, and how many of them are its first and its latest ones:
// the first rows come first, then the latest, then the rest by weight.
struct EvictSplit {
  int n, kept, first, last;
};
__device__ __forceinline__ EvictSplit evict_split(const KvView& kv, const int32_t* budget, int b, int b_max,
                                                  int n_sink, int n_recent) {
  EvictSplit s;
  s.n = paged_len(kv.seq_len, b, kv.max_len);
  s.kept = min(s.n, paged_len(budget, b, b_max));
  s.first = min(n_sink, s.kept);
  s.last = min(n_recent, s.kept - s.first);
  return s;
}

constexpr int EVS_THREADS = 512;
constexpr int EVS_MAX_CS = 16;
constexpr int EVS_SHARE_KEYS = 24576;          // staged keys up to which two CTAs share an SM
constexpr int EVS_UNROLL = 4;
constexpr int EVS_STAGE_KEYS = 49152;          // candidate keys a CTA stages (192 KB)

// One cluster of CS CTAs per (sequence, KV head).
template <int CS>
__global__ void __cluster_dims__(CS, 1, 1) __launch_bounds__(EVS_THREADS)
evict_select_kernel(const float* __restrict__ record, const KvView kv, const int32_t* __restrict__ budget,
                    int h_kv, int b_max, int n_sink, int n_recent, int32_t* __restrict__ idx_out,
                    int32_t* __restrict__ new_len) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ SelectSmem sm;
  extern __shared__ uint32_t staged[];

  const int rank = (int)cluster.block_rank();
  const int head = blockIdx.x / CS;
  const int b = head / h_kv, g = head - b * h_kv;
  const EvictSplit s = evict_split(kv, budget, b, b_max, n_sink, n_recent);
  int32_t* out = idx_out + (size_t)head * b_max;
  const int t0 = rank * blockDim.x + threadIdx.x, stride = CS * blockDim.x;
  if (g == 0 && t0 == 0) new_len[b] = s.kept;
  for (int i = s.kept + t0; i < b_max; i += stride) out[i] = -1;
  if (s.kept == s.n) {                         // everything stays
    for (int i = t0; i < s.n; i += stride) out[i] = i;
    return;
  }
  for (int i = t0; i < s.first; i += stride) out[i] = i;
  for (int i = t0; i < s.last; i += stride) out[s.kept - s.last + i] = s.n - s.last + i;
  const int take = s.kept - s.first - s.last;  // of the n - first - last candidates (more than take)
  if (take == 0) return;

  const int cand = s.n - s.first - s.last;
  const int per = (cand + CS - 1) / CS;
  const int lo = min(cand, rank * per), hi = min(cand, lo + per);
  // The slice's weights as ordered keys; NaN ranks with -inf, behind every number.  Positions
  // 4 i .. 4 i + 3 share a page: one table entry and one 16-byte load for four keys, and
  // EVS_UNROLL such groups in flight per thread.
  const int p0 = s.first + lo, p1 = s.first + hi;
  for (int i0 = p0 / 4 + threadIdx.x; 4 * i0 < p1; i0 += EVS_UNROLL * blockDim.x) {
    long long row[EVS_UNROLL];
#pragma unroll
    for (int u = 0; u < EVS_UNROLL; ++u) {
      const int j = 4 * (i0 + u * (int)blockDim.x);
      row[u] = j < p1 ? paged_row(kv, b, g, h_kv, j) : -1;
    }
    float4 w[EVS_UNROLL];
#pragma unroll
    for (int u = 0; u < EVS_UNROLL; ++u)
      w[u] = row[u] < 0 ? make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY)
                        : __ldg(reinterpret_cast<const float4*>(record + row[u]));
#pragma unroll
    for (int u = 0; u < EVS_UNROLL; ++u) {
      const int j = 4 * (i0 + u * (int)blockDim.x);
      const float x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e >= p0 && j + e < p1) staged[j + e - p0] = float_to_ordered(x[e] == x[e] ? x[e] : -INFINITY);
    }
  }
  __syncthreads();
  auto key_at = [&](int j) { return staged[j - lo]; };
  const SelectThreshold th = cluster_threshold<CS, true>(cluster, sm, key_at, lo, hi, take);
  ordered_emit<true>(sm, key_at, lo, hi, th, [&](int pos, int j) {
    if (pos < take) out[s.first + pos] = s.first + j;
    else flag_error(ERR_BAD_INDEX);            // unreachable when the counts are consistent
  });
  cluster_wait();                              // peers' last reads of this CTA's histograms
}

// Kept row i of (b, g), position idx[i], to position i of dst (its own table).  A warp takes 32
// rows: lane l looks up where row l lies and goes, then the rows' 16-byte vectors are copied
// with EVC_UNROLL loads each of K and V in flight per lane.  Bound by the rows' bytes: 32
// sequences of 8 KV heads, 1984 rows each of 256 + 256 bytes (520 MB moved), take 86 us (6.0
// TB/s); with a lookup per vector and one load in flight it was 121.
constexpr int EVC_WARPS = 8;
constexpr int EVC_UNROLL = 8;

template <int VPR>                             // 16-byte vectors per row
__global__ void __launch_bounds__(EVC_WARPS * 32)
evict_copy_kernel(uint4* __restrict__ k, uint4* __restrict__ v, float* __restrict__ record, const KvView kv,
                  const KvView dst, const int32_t* __restrict__ idx, const int32_t* __restrict__ new_len,
                  int h_kv, int b_max) {
  ptx::wait_dependency();
  const int head = blockIdx.x;
  const int b = head / h_kv, g = head - b * h_kv;
  const int lane = threadIdx.x & 31;
  const int kept = new_len[b];
  const int i0 = (blockIdx.y * EVC_WARPS + (threadIdx.x >> 5)) * 32;
  if (i0 >= kept) return;
  int from = -1, to = -1;                      // pools hold fewer than 2^31 rows
  if (i0 + lane < kept) {
    from = (int)paged_row(kv, b, g, h_kv, idx[(size_t)head * b_max + i0 + lane]);
    to = (int)paged_row(dst, b, g, h_kv, i0 + lane);
    if (from < 0) to = -1;
    if (to >= 0) record[to] = record[from];
  }
  // vector e of the 32 rows: row e / VPR
#pragma unroll 1
  for (int e0 = 0; e0 < VPR; e0 += EVC_UNROLL) {
    uint4 kx[EVC_UNROLL], vx[EVC_UNROLL];
    int at[EVC_UNROLL];
#pragma unroll
    for (int u = 0; u < EVC_UNROLL; ++u) {
      const int e = (e0 + u) * 32 + lane, vec = e % VPR;
      const int f = __shfl_sync(0xffffffffu, from, e / VPR);
      at[u] = __shfl_sync(0xffffffffu, to, e / VPR);
      if (at[u] >= 0) {
        kx[u] = __ldcs(k + (size_t)f * VPR + vec);
        vx[u] = __ldcs(v + (size_t)f * VPR + vec);
      }
    }
#pragma unroll
    for (int u = 0; u < EVC_UNROLL; ++u) {
      const int vec = ((e0 + u) * 32 + lane) % VPR;
      if (at[u] >= 0) {
        __stcs(k + (size_t)at[u] * VPR + vec, kx[u]);
        __stcs(v + (size_t)at[u] * VPR + vec, vx[u]);
      }
    }
  }
}

}  // namespace quoka
