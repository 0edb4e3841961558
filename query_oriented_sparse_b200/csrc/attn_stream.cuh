// Attention of one new token per sequence over its whole cache or a window of it, for a
// paged or a contiguous cache: out = softmax(q . k^T / sqrt(d)) . v over the visible keys
// j < n with j < n_sink or j >= n - window, n the sequence's tokens.
//
// The keys are read once and little is computed with each, so the kernel is bound by HBM.
// What matters is that every SM reads all the time, whatever the batch looks like.  So
// the work is cut by bytes, not by sequence: the visible keys of every (sequence, KV head)
// are counted in 128-key tiles, and CTA c of N takes tiles [c T / N, (c+1) T / N) of the
// list of all T, crossing sequences where the cut falls.  The lengths are read on the
// device, so a captured graph serves growing sequences.  A (sequence, KV head) that one
// CTA holds whole is finished there; one that several share leaves at most one partial
// (running maximum, sum and output, fp32) per CTA, two slots in all, and the join kernel
// merges them.  Where the sequences are short (four tiles at most), a CTA takes a (sequence,
// KV head) whole instead, and there is nothing to join: one launch.  With a weight record,
// the logits are kept (fp32, base 2) and the record kernel adds each key's softmax weight,
// summed over the group's heads, once the join has the row's maximum and sum.
//
// A sum of 0 stands for "no visible key" in partials, joins and results (such a row is zeros).  Keys
// that are there but whose logits are all -infinity leave a maximum of -infinity and no weight
// either, so their sum is set to 1: beside a finite maximum it weighs nothing, and alone it gives
// the NaN of 0 / 0, as in the chunk kernels.
//
// This file: the split, the CUDA-core kernel (fp32), the join and the record kernel.  fp32 with
// one head to a group reads at 5.8 TB/s (d 128, 16 sequences of 4K to 8K tokens); more heads
// make it wait for the logits' shared-memory reads (4 heads: 3.7 TB/s).
#pragma once
#include "attn_window.cuh"
#include "kv_pages.cuh"
#include "tc_ptx.cuh"

namespace quoka {

constexpr int AST_TILE = 128;             // keys per tile

// Visible key tiles of one sequence: nst tiles of first tokens, then tiles wt0 onwards.
struct KeySpan {
  int n, ns, lo;                          // visible: j < n and (j < ns or j >= lo)
  int nst, wt0, nt;

  __device__ __forceinline__ bool visible(int j) const { return j < n && (j < ns || j >= lo); }
  __device__ __forceinline__ int tile(int i) const { return i < nst ? i : i - nst + wt0; }
};

// An empty sequence has one tile without visible keys, so its (zero) output is written.
__device__ __forceinline__ KeySpan key_span(int n, int window, int n_sink) {
  KeySpan s;
  s.n = n;
  s.ns = min(n_sink, n);
  s.lo = max(0, n - window);
  if (s.ns >= s.lo) s.ns = s.lo = 0;
  s.nst = (s.ns + AST_TILE - 1) / AST_TILE;
  s.wt0 = max(s.lo / AST_TILE, s.nst);
  s.nt = max(1, s.nst + (n + AST_TILE - 1) / AST_TILE - s.wt0);
  return s;
}

struct StreamParams {
  KvView kv;
  int batch, h_q, h_kv, G;
  int window, n_sink;
  float scale_log2;                       // log2(e) / sqrt(d)
  int ctas;                               // N at most (the tiles, when they are fewer)
  int by_unit;                            // CTA c takes the whole (sequence, KV head) c: nothing to join
  int own_record;                         // and adds its keys' weights itself
  float* part;                            // [2 N][G][D] partial outputs
  float* part_ml;                         // [2 N][G][2] their running maximum (base 2) and sum
  float* unit_ml;                         // [batch * h_kv][G][2] maximum and 1 / sum (with a record)
  float* logits;                          // [tile][128][G] or NULL
  float* record;
};

template <bool kPaged>
__device__ __forceinline__ int stream_len(const StreamParams& p, const SeqTable& tab, int b) {
  if constexpr (kPaged) return paged_len(p.kv.seq_len, b, p.kv.max_len);
  else return tab.prefix[b] + 1;
}

// base[b] = tiles of one KV head of the sequences before b, from their lengths; base[batch]
// the total.  Every thread of the block calls it; it ends with a block barrier.
__device__ void stream_bases_of(const StreamParams& p, const int* lens, int* base) {
  if (threadIdx.x == 0) base[0] = 0;
  if (threadIdx.x < 32) {
    int run = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + threadIdx.x;
      int x = b < p.batch ? key_span(lens[b], p.window, p.n_sink).nt : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)threadIdx.x >= o) x += y;
      }
      x += run;
      if (b < p.batch) base[b + 1] = x;
      run = __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
}
// As above, reading the lengths first: lens and base are the block's shared memory.
template <bool kPaged>
__device__ void stream_bases(const StreamParams& p, const SeqTable& tab, int* lens, int* base) {
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) lens[b] = stream_len<kPaged>(p, tab, b);
  __syncthreads();
  stream_bases_of(p, lens, base);
}

__device__ __forceinline__ int stream_start(int c, int ctas, int tiles) {
  return (int)((long long)c * tiles / ctas);
}
__device__ __forceinline__ int stream_cta(int tile, int ctas, int tiles) {
  return (int)((((long long)tile + 1) * ctas - 1) / tiles);
}
// Sequence that tile x of the list belongs to.
__device__ __forceinline__ int stream_seq(const int* base, int batch, int h_kv, int x) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)base[mid] * h_kv <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tiles [x0, x1) of CTA c.
__device__ __forceinline__ void stream_share(const StreamParams& p, const int* base, int c, int* x0, int* x1) {
  const int tiles = base[p.batch] * p.h_kv;
  if (p.by_unit) {
    const int b = c / p.h_kv, nt = base[b + 1] - base[b];
    *x0 = base[b] * p.h_kv + (c - b * p.h_kv) * nt;
    *x1 = *x0 + nt;
    return;
  }
  const int ctas = min(p.ctas, tiles);                     // every share holds a tile at least
  *x0 = c < ctas ? stream_start(c, ctas, tiles) : 0;
  *x1 = c < ctas ? stream_start(c + 1, ctas, tiles) : 0;
}

// A run of tiles of one (sequence, KV head) inside a CTA's share.
struct StreamSeg {
  int b, g, unit, i0, cnt;                // tiles i0 .. i0 + cnt - 1 of the unit's nt
  bool whole;
  KeySpan span;
};
__device__ __forceinline__ StreamSeg stream_seg_of(const StreamParams& p, const int* lens, const int* base, int x,
                                                   int x1) {
  StreamSeg s;
  s.b = stream_seq(base, p.batch, p.h_kv, x);
  s.span = key_span(lens[s.b], p.window, p.n_sink);
  const int r = x - base[s.b] * p.h_kv;
  s.g = r / s.span.nt;
  s.i0 = r - s.g * s.span.nt;
  s.unit = s.b * p.h_kv + s.g;
  s.cnt = min(s.span.nt - s.i0, x1 - x);
  s.whole = s.cnt == s.span.nt;
  return s;
}

// Row of position j in the K/V pools or cache, -1 for none.
template <bool kPaged>
__device__ __forceinline__ long long stream_row(const StreamParams& p, const SeqTable& tab, int b, int g, int j) {
  if constexpr (kPaged) return paged_row(p.kv, b, g, p.h_kv, j);
  else return (long long)g * p.kv.rows_per_head + tab.kv_off[b] + j;
}

// record[key] += sum over the group's heads of 2^(s - M) / L for key j of segment sg, whose logits
// lie at lg.
__device__ __forceinline__ void stream_record_key(const StreamParams& p, const StreamSeg& sg, int j, const float* lg) {
  if (!sg.span.visible(j)) return;
  const float* ml = p.unit_ml + (size_t)sg.unit * p.G * 2;
  float w = 0.f;
  for (int r = 0; r < p.G; ++r) w += exp2f(lg[r] - ml[2 * r]) * ml[2 * r + 1];
  const long long row = paged_row(p.kv, sg.b, sg.g, p.h_kv, j);
  if (row >= 0) atomicAdd(p.record + row, w);
}

// A row's output element from its sum of p v, maximum and sum: zero without a visible key, NaN where
// every visible logit is -infinity.
__device__ __forceinline__ float stream_result(float o, float M, float L) {
  return L == 0.f ? 0.f : M == -INFINITY ? NAN : o / L;
}

template <typename T, int D, int R>
constexpr int ast_smem_bytes(int batch) {
  return adc_smem_bytes<T, D, R>() + (2 * batch + 1) * 4;
}

// CUDA-core form (fp32).  Warps take 32-key batches of the CTA's tiles in turn, each with
// its own stage in shared memory: lane l owns key l for the logits, then head dims
// [EPL l, EPL l + EPL) for P.V, as in attn_decode.cuh.  Rows of keys that are not visible
// are filled with zeros instead of read.  blockIdx.y: query heads R y .. of each group.
template <typename T, int D, int R, bool kPaged>
__global__ void __launch_bounds__(AdcCfg<T, D>::THREADS)
attn_stream_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                   const __grid_constant__ StreamParams p, const __grid_constant__ SeqTable tab,
                   T* __restrict__ out) {
  using Cfg = AdcCfg<T, D>;
  constexpr int NW = Cfg::NW, ROW = Cfg::ROW, VPR = Cfg::VPR, EPV = Cfg::EPV, EPL = Cfg::EPL;
  extern __shared__ __align__(16) unsigned char smem[];
  ptx::launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* qs = reinterpret_cast<float*>(smem);              // [R][D], times scale * log2(e)
  float* mls = qs + R * D;                                 // [NW][R][2]
  unsigned char* stage = smem + (R * D + NW * R * 2) * 4 + warp * (Cfg::STAGE + 32 * R * 4);
  unsigned char* vstage = stage + 32 * ROW;
  float* ps = reinterpret_cast<float*>(stage + Cfg::STAGE);
  int* base = reinterpret_cast<int*>(smem + adc_smem_bytes<T, D, R>());
  int* lens = base + p.batch + 1;
  stream_bases<kPaged>(p, tab, lens, base);

  const int c = blockIdx.x, r0 = blockIdx.y * R;
  const int rows = min(R, p.G - r0);
  int x0, x1;
  stream_share(p, base, c, &x0, &x1);
  for (int x = x0; x < x1;) {
    const StreamSeg sg = stream_seg_of(p, lens, base, x, x1);
    for (int e = threadIdx.x; e < R * D; e += blockDim.x) {
      const int r = e / D, d = e - r * D;
      qs[e] = r < rows ? to_f32(q[((size_t)sg.b * p.h_q + (size_t)sg.g * p.G + r0 + r) * D + d]) * p.scale_log2 : 0.f;
    }
    __syncthreads();
    float m[R], l[R], acc[R][EPL];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[r][e] = 0.f;
    }
    bool seen = false;                                     // a visible key so far
    for (int w = warp; w < sg.cnt * 4; w += NW) {          // 32-key batches of the segment
      const int j = sg.span.tile(sg.i0 + (w >> 2)) * AST_TILE + (w & 3) * 32 + lane;
      bool vis = sg.span.visible(j);
      int row = 0;
      if (vis) {
        const long long rr = stream_row<kPaged>(p, tab, sg.b, sg.g, j);
        row = rr < 0 ? 0 : (int)rr;                        // pools and caches hold fewer than 2^31 rows
        if (rr < 0) vis = false;
      }
      const unsigned on = __ballot_sync(0xffffffffu, vis);
      float sc[R];
      if (on) {
#pragma unroll 4
        for (int e = lane; e < 32 * VPR; e += 32) {
          const int kk = e / VPR, vv = e - kk * VPR;
          const int rk = __shfl_sync(0xffffffffu, row, kk);
          adc_cp16z(stage + kk * ROW + vv * 16, k + (size_t)rk * D + vv * EPV, (on >> kk) & 1u);
        }
        adc_commit();
#pragma unroll 4
        for (int e = lane; e < 32 * VPR; e += 32) {
          const int kk = e / VPR, vv = e - kk * VPR;
          const int rk = __shfl_sync(0xffffffffu, row, kk);
          adc_cp16z(vstage + kk * ROW + vv * 16, v + (size_t)rk * D + vv * EPV, (on >> kk) & 1u);
        }
        adc_commit();
        adc_wait<1>();
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) sc[r] = 0.f;
        const unsigned char* krow = stage + lane * ROW;
#pragma unroll 2
        for (int cc = 0; cc < VPR; ++cc) {
          float kx[EPV];
          smem_vec16<T>(krow + cc * 16, kx);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float* qr = qs + r * D + cc * EPV;
#pragma unroll
            for (int e4 = 0; e4 < EPV; e4 += 4) {
              const float4 qv = *reinterpret_cast<const float4*>(qr + e4);
              sc[r] = fmaf(qv.x, kx[e4], sc[r]);
              sc[r] = fmaf(qv.y, kx[e4 + 1], sc[r]);
              sc[r] = fmaf(qv.z, kx[e4 + 2], sc[r]);
              sc[r] = fmaf(qv.w, kx[e4 + 3], sc[r]);
            }
          }
        }
      }
      if (!vis) {
#pragma unroll
        for (int r = 0; r < R; ++r) sc[r] = -INFINITY;
      }
      if (p.logits) {
        float* lg = p.logits + ((size_t)(x + (w >> 2)) * AST_TILE + (w & 3) * 32 + lane) * p.G + r0;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < rows) lg[r] = sc[r];
      }
      if (!on) continue;
      seen = true;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float mx = sc[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[r], mx);
        // (a maximum of -inf: the keys so far are masked and weigh 0, or NaN, which stays)
        const float pr = exp2f(sc[r] - (mn == -INFINITY ? 0.f : mn));
        const float corr = mn == -INFINITY ? 1.f : exp2f(m[r] - mn);
        float sum = pr;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[r] = l[r] * corr + sum;
        m[r] = mn;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[r][e] *= corr;
        ps[lane * R + r] = pr;
      }
      adc_wait<0>();
      __syncwarp();
      for (int kk = 0; kk < 32; ++kk) {
        float vx[EPL];
        smem_vecn<T, EPL>(vstage + kk * ROW + lane * EPL * Cfg::ESZ, vx);
        const float* pk = ps + kk * R;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float pr = pk[r];
#pragma unroll
          for (int e = 0; e < EPL; ++e) acc[r][e] = fmaf(pr, vx[e], acc[r][e]);
        }
      }
      __syncwarp();                                        // stage free for the next batch
    }

    // merge the warps of the CTA
    float* wout = reinterpret_cast<float*>(stage);
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        mls[(warp * R + r) * 2] = m[r];
        mls[(warp * R + r) * 2 + 1] = seen && l[r] == 0.f ? 1.f : l[r];
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < EPL; ++e) wout[r * D + lane * EPL + e] = acc[r][e];
    __syncthreads();
    const int slot = 2 * c + (x == x0 ? 0 : 1);
    for (int e = threadIdx.x; e < rows * D; e += blockDim.x) {
      const int r = e / D, d = e - r * D;
      float M = -INFINITY, L = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, mls[(w * R + r) * 2]);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float mw = mls[(w * R + r) * 2], lw = mls[(w * R + r) * 2 + 1];
        const float* ww = reinterpret_cast<const float*>(smem + (R * D + NW * R * 2) * 4 +
                                                         w * (Cfg::STAGE + 32 * R * 4));
        if (lw != 0.f) {                                   // a warp without visible keys adds nothing
          const float f = M == -INFINITY ? 1.f : exp2f(mw - M);
          o = fmaf(ww[e], f, o);
          L = fmaf(lw, f, L);
        }
      }
      if (sg.whole) {
        out[((size_t)sg.b * p.h_q + (size_t)sg.g * p.G + r0 + r) * D + d] = from_f32<T>(stream_result(o, M, L));
        if (d == 0 && p.logits) {
          p.unit_ml[((size_t)sg.unit * p.G + r0 + r) * 2] = M;
          p.unit_ml[((size_t)sg.unit * p.G + r0 + r) * 2 + 1] = L == 0.f ? 0.f : 1.f / L;
        }
      } else {
        p.part[((size_t)slot * p.G + r0 + r) * D + d] = o;
        if (d == 0) {
          p.part_ml[((size_t)slot * p.G + r0 + r) * 2] = M;
          p.part_ml[((size_t)slot * p.G + r0 + r) * 2 + 1] = L;
        }
      }
    }
    __syncthreads();                                       // qs, mls and the stages are free; unit_ml is there
    if (kPaged && p.own_record)
      for (int e = threadIdx.x; e < sg.cnt * AST_TILE; e += blockDim.x)
        stream_record_key(p, sg, sg.span.tile(sg.i0 + e / AST_TILE) * AST_TILE + e % AST_TILE,
                          p.logits + ((size_t)x * AST_TILE + e) * p.G);
    x += sg.cnt;
  }
}

constexpr int ASJ_ROWS = 8;                // output rows (warps) per block of the join

// Slot of CTA c's partial of a unit whose tiles start at s: the CTA's first segment when
// its share starts inside the unit, else its last.
__device__ __forceinline__ int stream_slot(int c, int s, int ctas, int tiles) {
  return 2 * c + (stream_start(c, ctas, tiles) >= s ? 0 : 1);
}

// One warp per output row (sequence, query head): out = sum_c o_c 2^(m_c - M) / sum_c l_c 2^(m_c - M)
// over the CTAs that share its (sequence, KV head).  Launched as a programmatic dependent: its
// blocks work out their units while the streaming kernel still runs (1.5 to 2 us less per step).
template <typename T, int D, bool kPaged>
__global__ void __launch_bounds__(ASJ_ROWS * 32)
attn_stream_join_kernel(const __grid_constant__ StreamParams p, const __grid_constant__ SeqTable tab,
                        T* __restrict__ out) {
  extern __shared__ int base[];                            // [batch + 1], lengths [batch]
  ptx::launch_dependents();
  stream_bases<kPaged>(p, tab, base + p.batch + 1, base);
  ptx::wait_dependency();                                  // in every block: what follows this grid relies on it
  if (p.by_unit) return;                                   // nothing to join
  const int tiles = base[p.batch] * p.h_kv, ctas = min(p.ctas, tiles);
  const int row = blockIdx.x * ASJ_ROWS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= p.batch * p.h_q) return;
  const int unit = row / p.G, r = row - unit * p.G;
  const int b = unit / p.h_kv, g = unit - b * p.h_kv;
  const int nt = base[b + 1] - base[b];
  const int s = base[b] * p.h_kv + g * nt;
  const int c0 = stream_cta(s, ctas, tiles), nc = stream_cta(s + nt - 1, ctas, tiles) - c0 + 1;
  if (nc == 1) return;                                     // finished by its CTA
  auto part_row = [&](int i) { return (size_t)stream_slot(c0 + i, s, ctas, tiles) * p.G + r; };
  float M = -INFINITY, L = 0.f;
  for (int i = lane; i < nc; i += 32) {
    const float* ml = p.part_ml + part_row(i) * 2;
    if (ml[1] != 0.f) M = fmaxf(M, ml[0]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  constexpr int E = D / 32;                                // output elements per lane
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int i0 = 0; i0 < nc; i0 += 32) {
    // lane i: partial i0 + i and its weight (0 for one without visible keys, whose O is not read)
    const size_t mine = i0 + lane < nc ? part_row(i0 + lane) : 0;
    float f = 0.f;
    if (i0 + lane < nc) {
      const float ml = p.part_ml[mine * 2], ll = p.part_ml[mine * 2 + 1];
      f = ll != 0.f ? exp2f(ml - M) : 0.f;
      if (ll != 0.f) L = fmaf(ll, f, L);
    }
    const int lim = min(32, nc - i0);
    for (int i = 0; i < lim; i += 8) {
      float xs[8][E], fs[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const size_t pr = __shfl_sync(0xffffffffu, (unsigned long long)mine, (i + u) & 31);
        fs[u] = __shfl_sync(0xffffffffu, f, (i + u) & 31);
        if (i + u >= lim) fs[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) xs[u][e] = 0.f;
        if (fs[u] != 0.f) load_vec<float, E>(p.part + pr * D + lane * E, xs[u]);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fs[u] != 0.f ? fmaf(xs[u][e], fs[u], o[e]) : o[e];
    }
  }
  L = warp_sum(L);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  if (lane == 0 && p.logits) {
    p.unit_ml[(size_t)row * 2] = M;
    p.unit_ml[(size_t)row * 2 + 1] = inv;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[(size_t)row * D + lane * E + e] = from_f32<T>(o[e] * inv);
}

// One thread per key of a tile.
// The add is a reduction in memory, so a page that two sequences share gets both sums.
__global__ void __launch_bounds__(AST_TILE)
attn_stream_record_kernel(const __grid_constant__ StreamParams p, const __grid_constant__ SeqTable tab) {
  extern __shared__ int base[];                            // [batch + 1], lengths [batch]
  const int* lens = base + p.batch + 1;
  stream_bases<true>(p, tab, base + p.batch + 1, base);
  ptx::wait_dependency();
  const int tiles = base[p.batch] * p.h_kv;
  for (int x = blockIdx.x; x < tiles; x += gridDim.x) {
    const StreamSeg sg = stream_seg_of(p, lens, base, x, x + 1);
    stream_record_key(p, sg, sg.span.tile(sg.i0) * AST_TILE + threadIdx.x,
                      p.logits + ((size_t)x * AST_TILE + threadIdx.x) * p.G);
  }
}

}  // namespace quoka
