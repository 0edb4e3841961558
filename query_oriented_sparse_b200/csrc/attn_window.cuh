// Attention of a chunk over a sliding window of the contiguous cache and a few first
// tokens: query t (position p = P + t) sees key j <= p when j < n_sink or j > p - window.
//
// CUDA-core form, for fp32 (the 1e-4 relative bound rules out tf32 products).  A tile is 64
// query rows, the G query heads of a KV head at 64 / G positions each, so that short chunks
// fill it too.  One CTA walks the visible keys of a tile in blocks of 64: the first tokens, then
// the window from the first row's oldest key to the last row's own, with the online softmax in
// fp32; when the tiles are few, each tile's blocks are split over several CTAs, whose partials
// window_join_kernel merges.  It is bound by the FMAs and the shared-memory reads that feed
// them: a thread holds 4 x 4 logits and 4 x D/16 outputs and reads in 16-byte vectors along the
// summed axis (one read for eight FMAs; rows padded by 16 bytes, so that a quarter warp's reads
// hit all banks), which keeps the shared-memory pipe busy for three quarters of the FMAs' time;
// the next block's rows come in by cp.async meanwhile.  29.8 TFLOP/s, 40 % of the FMA rate, for
// 2048 queries through a window of 1024 keys at d 128, where scalar reads of single-buffered
// blocks gave 20.9.  Blocks that some row does not see whole are masked by selection, and P.V skips
// masked keys there, so that a value that is not a number reaches only the rows that see it.
#pragma once
#include "attn_decode.cuh"

namespace quoka {

// 16-byte asynchronous copy, or 16 zero bytes when `on` is false (nothing is read then).
__device__ __forceinline__ void adc_cp16z(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(on ? 16 : 0)
               : "memory");
}

// Visible keys of the query positions [p0, p1] (absolute): first tokens [0, ns), then
// [w0, p1].  ns is 0 when the two join.
struct WindowSpan {
  int ns, w0, p1;
};
__device__ __forceinline__ WindowSpan window_span(int p0, int p1, int window, int n_sink) {
  WindowSpan s;
  s.p1 = p1;
  s.w0 = max(0, p0 - window + 1);
  s.ns = min(n_sink, p1 + 1);
  if (s.ns >= s.w0) {
    s.ns = 0;
    s.w0 = 0;
  }
  return s;
}

constexpr int AWS_ROWS = 64;
constexpr int AWS_KEYS = 64;
constexpr int AWS_THREADS = 256;

struct WindowParams {
  int h_q, h_kv, G, C, TP, window, n_sink;   // TP: positions per query head and tile (of one CTA)
  int nsplit;                      // units per tile
  long long rows_per_head;
  float scale_log2;                // log2(e) / sqrt(d)
  float* part;                     // [tile][unit][rows of the tile][D], then
  float* part_ml;                  // [tile][unit][rows of the tile][2], when nsplit > 1
};

template <int D>
struct AwsCfg {
  static constexpr int LD = D + 4;                    // padded row, floats
  static constexpr int LP = AWS_KEYS + 4;
  static constexpr int KV = AWS_KEYS * (LD + D);      // one block's K and V
  static constexpr int SMEM = (AWS_ROWS * LD + 2 * KV + AWS_ROWS * LP) * 4;
};

template <int D>
__global__ void __launch_bounds__(AWS_THREADS)
window_simt_kernel(const float* __restrict__ q, const float* __restrict__ k_cache, const float* __restrict__ v_cache,
                   const __grid_constant__ SeqTable tab, const __grid_constant__ WindowParams p,
                   float* __restrict__ out) {
  using Cfg = AwsCfg<D>;
  constexpr int LD = Cfg::LD, LP = Cfg::LP;
  constexpr int DJ = D / 64;                          // output columns per thread: 4 at tc * 4 + 64 j
  extern __shared__ __align__(16) float smem_f[];
  float* Qs = smem_f;
  float* KVs = Qs + AWS_ROWS * LD;                    // [2][K rows padded, V rows]
  float* Ps = KVs + 2 * Cfg::KV;

  const int ntp = (p.C + p.TP - 1) / p.TP;
  const int tile = blockIdx.x / p.nsplit, part = blockIdx.x - tile * p.nsplit;
  const int t0 = (ntp - 1 - tile % ntp) * p.TP;       // longest key ranges first
  const int b = tile / ntp / p.h_kv, g = tile / ntp - b * p.h_kv;
  const int P = tab.prefix[b], C = p.C, window = p.window, n_sink = p.n_sink;
  const int tid = threadIdx.x, tc = tid & 15, tr = tid >> 4;
  const WindowSpan sp = window_span(P + t0, P + min(C, t0 + p.TP) - 1, window, n_sink);
  const int nsb = (sp.ns + AWS_KEYS - 1) / AWS_KEYS;
  const int nblk = nsb + (sp.p1 - sp.w0) / AWS_KEYS + 1;
  const int blk0 = (int)((long long)nblk * part / p.nsplit), blk1 = (int)((long long)nblk * (part + 1) / p.nsplit);
  const size_t head_row0 = (size_t)g * p.rows_per_head + tab.kv_off[b];
  const float* kh = k_cache + head_row0 * D;
  const float* vh = v_cache + head_row0 * D;
  // row r: head g G + r / TP at position t0 + r % TP; its place in q and out, -1 for none
  auto row_at = [&](int r) {
    const int hl = r / p.TP, t = t0 + r - hl * p.TP;
    return hl < p.G && t < C ? (b * p.h_q + g * p.G + hl) * C + t : -1;
  };

  auto start = [&](int blk) { return blk < nsb ? blk * AWS_KEYS : sp.w0 + (blk - nsb) * AWS_KEYS; };
  auto limit = [&](int blk) { return min(AWS_KEYS, (blk < nsb ? sp.ns : sp.p1 + 1) - start(blk)); };
  auto fetch = [&](int blk) {                         // rows past the block's limit become zero
    float* Ks = KVs + (blk & 1) * Cfg::KV;
    float* Vs = Ks + AWS_KEYS * LD;
    const int j0 = start(blk), n = limit(blk);
    for (int e = tid; e < AWS_KEYS * (D / 4); e += AWS_THREADS) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      const size_t src = (size_t)(j0 + (r < n ? r : 0)) * D + c;
      adc_cp16z(Ks + r * LD + c, kh + src, r < n);
      adc_cp16z(Vs + r * D + c, vh + src, r < n);
    }
    adc_commit();
  };

  for (int e = tid; e < AWS_ROWS * (D / 4); e += AWS_THREADS) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    const int at = row_at(r);
    adc_cp16z(Qs + r * LD + c, q + (size_t)max(at, 0) * D + c, at >= 0);
  }
  if (blk0 < blk1) {
    fetch(blk0);
  } else {
    adc_commit();
    adc_wait<0>();
  }

  float m[4], l[4], o[4][DJ][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < DJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
  }

  int pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pos[i] = P + t0 + (tr + 16 * i) % p.TP;
  for (int blk = blk0; blk < blk1; ++blk) {
    const float* Ks = KVs + (blk & 1) * Cfg::KV;
    const float* Vs = Ks + AWS_KEYS * LD;
    const int j0 = start(blk), klim = limit(blk);
    // every row sees every key of the block (rows past C are not written)
    const bool whole = klim == AWS_KEYS && (blk < nsb || (j0 + AWS_KEYS - 1 <= P + t0 && j0 > sp.p1 - window));
    if (blk + 1 < blk1) {
      fetch(blk + 1);                                 // (its stage was released by the barrier below)
      adc_wait<1>();
    } else {
      adc_wait<0>();
    }
    __syncthreads();

    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 qv[4], kv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(Qs + (tr + 16 * i) * LD + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tc + 16 * j) * LD + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
          s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
          s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
          s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
        }
    }

    float al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float rmax = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kk = j0 + tc + 16 * j;
        const bool ok = whole || (tc + 16 * j < klim && kk <= pos[i] && (kk < n_sink || kk > pos[i] - window));
        s[i][j] = ok ? s[i][j] * p.scale_log2 : -INFINITY;
        rmax = fmaxf(rmax, s[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) rmax = fmaxf(rmax, __shfl_xor_sync(0xffffffffu, rmax, off));
      const float mnew = fmaxf(m[i], rmax);
      const float muse = (mnew == -INFINITY) ? 0.f : mnew;
      al[i] = exp2f(m[i] - muse);
      float rsum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float pr = exp2f(s[i][j] - muse);
        rsum += pr;
        Ps[(tr + 16 * i) * LP + tc + 16 * j] = pr;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) rsum += __shfl_xor_sync(0xffffffffu, rsum, off);
      l[i] = l[i] * al[i] + rsum;
      m[i] = mnew;
    }
    __syncwarp();                                     // a row's weights are written and read by one warp
    // the block's P.V is summed by itself, so that no sum runs over more than 64 keys or over
    // the blocks
    float ob[4][DJ][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < DJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) ob[i][j][e] = 0.f;
    for (int kk = 0; kk < klim; kk += 4) {
      float4 pv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4*>(Ps + (tr + 16 * i) * LP + kk);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float4 vv[DJ];
#pragma unroll
        for (int j = 0; j < DJ; ++j) vv[j] = *reinterpret_cast<const float4*>(Vs + (kk + u) * D + tc * 4 + 64 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float pr = u == 0 ? pv[i].x : u == 1 ? pv[i].y : u == 2 ? pv[i].z : pv[i].w;
          if (!whole && pr == 0.f) continue;
#pragma unroll
          for (int j = 0; j < DJ; ++j) {
            ob[i][j][0] = fmaf(pr, vv[j].x, ob[i][j][0]);
            ob[i][j][1] = fmaf(pr, vv[j].y, ob[i][j][1]);
            ob[i][j][2] = fmaf(pr, vv[j].z, ob[i][j][2]);
            ob[i][j][3] = fmaf(pr, vv[j].w, ob[i][j][3]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < DJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] = fmaf(o[i][j][e], al[i], ob[i][j][e]);
    __syncthreads();                                  // the block's stage and Ps are free
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = tr + 16 * i, at = row_at(r);
    if (at < 0) continue;
    const size_t prow = (size_t)blockIdx.x * AWS_ROWS + r;
    const bool split = p.nsplit > 1;
    if (split && tc == 0) {
      p.part_ml[prow * 2] = m[i];
      p.part_ml[prow * 2 + 1] = l[i];
    }
    const float inv = split ? 1.f : 1.0f / l[i];      // every row sees at least its own key
    float* dst = split ? p.part + prow * D : out + (size_t)at * D;
#pragma unroll
    for (int j = 0; j < DJ; ++j)
      *reinterpret_cast<float4*>(dst + tc * 4 + 64 * j) =
          make_float4(o[i][j][0] * inv, o[i][j][1] * inv, o[i][j][2] * inv, o[i][j][3] * inv);
  }
}

// Joins the units of each tile: out = sum_u O_u 2^(m_u - M) / sum_u l_u 2^(m_u - M).  One thread
// per 8 output columns.  CTAS CTAs of ROWS rows to a tile.
constexpr int AWJ_THREADS = 256;
template <typename T, int D, int CTAS, int ROWS>
__global__ void __launch_bounds__(AWJ_THREADS)
window_join_kernel(const __grid_constant__ WindowParams p, long long total, T* __restrict__ out) {
  constexpr int VPR = D / 8;
  const long long e = (long long)blockIdx.x * AWJ_THREADS + threadIdx.x;
  if (e >= total) return;
  const long long row = e / VPR;           // (b * h_q + h) * C + t
  const int c = (int)(e - row * VPR) * 8;
  const int t = (int)(row % p.C);
  const long long bh = row / p.C;
  const int b = (int)(bh / p.h_q), h = (int)(bh - (long long)b * p.h_q);
  const int g = h / p.G, hl = h - g * p.G;
  const int span = CTAS * p.TP, ntp = (p.C + span - 1) / span;
  const int in = t % span, rank = in / p.TP;
  const long long tile = ((long long)b * p.h_kv + g) * ntp + (ntp - 1 - t / span);
  const size_t r0 = ((size_t)tile * p.nsplit * CTAS + rank) * ROWS + hl * p.TP + in % p.TP;
  const size_t step = (size_t)CTAS * ROWS;
  float M = -INFINITY, L = 0.f, o[8];
  for (int s = 0; s < p.nsplit; ++s)
    if (p.part_ml[(r0 + s * step) * 2 + 1] != 0.f) M = fmaxf(M, p.part_ml[(r0 + s * step) * 2]);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  for (int s = 0; s < p.nsplit; ++s) {
    const float l = p.part_ml[(r0 + s * step) * 2 + 1];
    if (l == 0.f) continue;                // no visible key: its O is not set
    const float f = exp2f(p.part_ml[(r0 + s * step) * 2] - M);
    L = fmaf(l, f, L);
    const float4* src = reinterpret_cast<const float4*>(p.part + (r0 + s * step) * D + c);
    const float4 a = src[0], d = src[1];
    o[0] = fmaf(a.x, f, o[0]); o[1] = fmaf(a.y, f, o[1]); o[2] = fmaf(a.z, f, o[2]); o[3] = fmaf(a.w, f, o[3]);
    o[4] = fmaf(d.x, f, o[4]); o[5] = fmaf(d.y, f, o[5]); o[6] = fmaf(d.z, f, o[6]); o[7] = fmaf(d.w, f, o[7]);
  }
  const float inv = 1.f / L;
  __align__(16) T y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = from_f32<T>(o[i] * inv);
#pragma unroll
  for (int i = 0; i < (int)sizeof(y) / 16; ++i)
    reinterpret_cast<uint4*>(out + e * 8)[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(y) + 16 * i);
}

}  // namespace quoka
