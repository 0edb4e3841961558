// Attention of a chunk over a sliding window of the contiguous cache and a few first
// tokens: query t (position p = P + t) sees key j <= p when j < n_sink or j > p - window.
//
// CUDA-core form, for fp32 (the 1e-4 relative bound rules out tf32 products).  One CTA per
// (sequence, query head, 64 query rows) walks the visible keys of its rows in blocks of 64:
// the first tokens, then the window from the first row's oldest key to the last row's own,
// with the online softmax in fp32.  It is bound by the FMA units, so a thread holds 4 x 4
// logits and 4 x D/16 outputs and reads shared memory in 16-byte vectors along the summed
// axis (one read for eight FMAs; rows padded by 16 bytes, so that a quarter warp's reads hit
// all banks), and the next block's rows come in by cp.async meanwhile: SIMTFIG.  Blocks that
// some row does not see whole are masked by selection, and P.V skips masked keys there, so
// that a value that is not a number reaches only the rows that see it.
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
                   long long rows_per_head, const __grid_constant__ SeqTable tab, int h_q, int h_kv, int C,
                   int window, int n_sink, float* __restrict__ out, float scale_log2) {
  using Cfg = AwsCfg<D>;
  constexpr int LD = Cfg::LD, LP = Cfg::LP;
  constexpr int DJ = D / 64;                          // output columns per thread: 4 at tc * 4 + 64 j
  extern __shared__ __align__(16) float smem_f[];
  float* Qs = smem_f;
  float* KVs = Qs + AWS_ROWS * LD;                    // [2][K rows padded, V rows]
  float* Ps = KVs + 2 * Cfg::KV;

  const int b = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * AWS_ROWS;
  const int G = h_q / h_kv, g = h / G;
  const int P = tab.prefix[b];
  const int tid = threadIdx.x, tc = tid & 15, tr = tid >> 4;
  const WindowSpan sp = window_span(P + t0, P + min(C, t0 + AWS_ROWS) - 1, window, n_sink);
  const int nsb = (sp.ns + AWS_KEYS - 1) / AWS_KEYS;
  const int nblk = nsb + (sp.p1 - sp.w0) / AWS_KEYS + 1;
  const size_t head_row0 = (size_t)g * rows_per_head + tab.kv_off[b];
  const float* kh = k_cache + head_row0 * D;
  const float* vh = v_cache + head_row0 * D;
  const float* qh = q + ((size_t)(b * h_q + h) * C) * D;

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
    adc_cp16z(Qs + r * LD + c, qh + (size_t)(t0 + r < C ? t0 + r : t0) * D + c, t0 + r < C);
  }
  fetch(0);

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

  for (int blk = 0; blk < nblk; ++blk) {
    const float* Ks = KVs + (blk & 1) * Cfg::KV;
    const float* Vs = Ks + AWS_KEYS * LD;
    const int j0 = start(blk), klim = limit(blk);
    // every row sees every key of the block (rows past C are not written)
    const bool whole = klim == AWS_KEYS && (blk < nsb || (j0 + AWS_KEYS - 1 <= P + t0 && j0 > sp.p1 - window));
    if (blk + 1 < nblk) {
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

#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = P + t0 + tr + 16 * i;
      float rmax = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kk = j0 + tc + 16 * j;
        const bool ok = whole || (tc + 16 * j < klim && kk <= pos && (kk < n_sink || kk > pos - window));
        s[i][j] = ok ? s[i][j] * scale_log2 : -INFINITY;
        rmax = fmaxf(rmax, s[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) rmax = fmaxf(rmax, __shfl_xor_sync(0xffffffffu, rmax, off));
      const float mnew = fmaxf(m[i], rmax);
      const float muse = (mnew == -INFINITY) ? 0.f : mnew;
      const float alpha = exp2f(m[i] - muse);
      float rsum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float pr = exp2f(s[i][j] - muse);
        rsum += pr;
        Ps[(tr + 16 * i) * LP + tc + 16 * j] = pr;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) rsum += __shfl_xor_sync(0xffffffffu, rsum, off);
      l[i] = l[i] * alpha + rsum;
      m[i] = mnew;
#pragma unroll
      for (int j = 0; j < DJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] *= alpha;
    }
    __syncwarp();                                     // a row's weights are written and read by one warp
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
            o[i][j][0] = fmaf(pr, vv[j].x, o[i][j][0]);
            o[i][j][1] = fmaf(pr, vv[j].y, o[i][j][1]);
            o[i][j][2] = fmaf(pr, vv[j].z, o[i][j][2]);
            o[i][j][3] = fmaf(pr, vv[j].w, o[i][j][3]);
          }
        }
      }
    }
    __syncthreads();                                  // the block's stage and Ps are free
  }

  float* oh = out + ((size_t)(b * h_q + h) * C) * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + tr + 16 * i;
    if (t < C) {
      const float inv = 1.0f / l[i];                  // every row sees at least its own key
#pragma unroll
      for (int j = 0; j < DJ; ++j)
        *reinterpret_cast<float4*>(oh + (size_t)t * D + tc * 4 + 64 * j) =
            make_float4(o[i][j][0] * inv, o[i][j][1] * inv, o[i][j][2] * inv, o[i][j][3] * inv);
    }
  }
}

}  // namespace quoka
