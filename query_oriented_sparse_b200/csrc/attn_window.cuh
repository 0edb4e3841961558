// Attention of a chunk over a sliding window of the contiguous cache and a few first
// tokens: query t (position p = P + t) sees key j <= p when j < n_sink or j > p - window.
//
// CUDA-core form, for fp32 (the 1e-4 relative bound rules out tf32 products).  One CTA per
// (sequence, query head, 64 query rows) walks the visible keys of its rows in blocks of 64:
// the first tokens, then the window from the first row's oldest key to the last row's own,
// with the online softmax in fp32.  Blocks that some row does not see whole are masked by
// selection, and P.V skips masked keys there, so that a value that is not a number reaches
// only the rows that see it.
#pragma once
#include "attn_simt.cuh"

namespace quoka {

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

template <typename T, int D>
__global__ void __launch_bounds__(ATS_THREADS)
window_simt_kernel(const T* __restrict__ q, const T* __restrict__ k_cache, const T* __restrict__ v_cache,
                   long long rows_per_head, const __grid_constant__ SeqTable tab, int h_q, int h_kv, int C,
                   int window, int n_sink, T* __restrict__ out, float scale_log2) {
  constexpr int LD = D + 1;
  constexpr int DJ = D / 16;                  // output columns per thread
  extern __shared__ __align__(16) unsigned char smem_raw[];
  float* Qs = reinterpret_cast<float*>(smem_raw);
  float* Ks = Qs + ATS_ROWS * LD;
  float* Vs = Ks + ATS_KEYS * LD;
  float* Ps = Vs + ATS_KEYS * D;

  const int b = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * ATS_ROWS;
  const int G = h_q / h_kv, g = h / G;
  const int P = tab.prefix[b];
  const int tid = threadIdx.x, tc = tid & 15, tr = tid >> 4;
  const WindowSpan sp = window_span(P + t0, P + min(C, t0 + ATS_ROWS) - 1, window, n_sink);
  const int nsb = (sp.ns + ATS_KEYS - 1) / ATS_KEYS;
  const int nblk = nsb + (sp.p1 - sp.w0) / ATS_KEYS + 1;
  const size_t head_row0 = (size_t)g * rows_per_head + tab.kv_off[b];
  const T* kh = k_cache + head_row0 * D;
  const T* vh = v_cache + head_row0 * D;
  const T* qh = q + ((size_t)(b * h_q + h) * C) * D;

  for (int e = tid * 4; e < ATS_ROWS * D; e += ATS_THREADS * 4) {
    const int r = e / D, c = e % D;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (t0 + r < C) load_vec<T, 4>(qh + (size_t)(t0 + r) * D + c, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) Qs[r * LD + c + i] = x[i];
  }

  float m[4], l[4], o[4][DJ];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < DJ; ++j) o[i][j] = 0.f;
  }

  for (int blk = 0; blk < nblk; ++blk) {
    const int j0 = blk < nsb ? blk * ATS_KEYS : sp.w0 + (blk - nsb) * ATS_KEYS;
    const int jend = blk < nsb ? sp.ns : sp.p1 + 1;        // keys [j0, min(j0 + 64, jend))
    const int klim = min(ATS_KEYS, jend - j0);
    // every row sees every key of the block (rows past C are not written)
    const bool whole = klim == ATS_KEYS && (blk < nsb || (j0 + ATS_KEYS - 1 <= P + t0 && j0 > sp.p1 - window));
    __syncthreads();                           // previous block fully consumed
    for (int e = tid * 4; e < ATS_KEYS * D; e += ATS_THREADS * 4) {
      const int r = e / D, c = e % D;
      float xk[4] = {0.f, 0.f, 0.f, 0.f}, xv[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < klim) {
        load_vec<T, 4>(kh + (size_t)(j0 + r) * D + c, xk);
        load_vec<T, 4>(vh + (size_t)(j0 + r) * D + c, xv);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Ks[r * LD + c + i] = xk[i];
        Vs[r * D + c + i] = xv[i];
      }
    }
    __syncthreads();

    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; ++d) {
      float qv[4], kv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qv[i] = Qs[(tr + 16 * i) * LD + d];
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = Ks[(tc + 16 * j) * LD + d];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = fmaf(qv[i], kv[j], s[i][j]);
    }

#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = P + t0 + tr + 16 * i;
      float rmax = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kk = j0 + tc + 16 * j;
        const bool ok = kk < jend && kk <= pos && (kk < n_sink || kk > pos - window);
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
        const float p = exp2f(s[i][j] - muse);
        rsum += p;
        Ps[(tr + 16 * i) * (ATS_KEYS + 1) + tc + 16 * j] = p;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) rsum += __shfl_xor_sync(0xffffffffu, rsum, off);
      l[i] = l[i] * alpha + rsum;
      m[i] = mnew;
#pragma unroll
      for (int j = 0; j < DJ; ++j) o[i][j] *= alpha;
    }
    __syncthreads();
    if (whole) {
#pragma unroll 4
      for (int kk = 0; kk < ATS_KEYS; ++kk) {
        float pv[4], vv[DJ];
#pragma unroll
        for (int i = 0; i < 4; ++i) pv[i] = Ps[(tr + 16 * i) * (ATS_KEYS + 1) + kk];
#pragma unroll
        for (int j = 0; j < DJ; ++j) vv[j] = Vs[kk * D + tc + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < DJ; ++j) o[i][j] = fmaf(pv[i], vv[j], o[i][j]);
      }
    } else {
      for (int kk = 0; kk < klim; ++kk) {
        float pv[4], vv[DJ];
#pragma unroll
        for (int i = 0; i < 4; ++i) pv[i] = Ps[(tr + 16 * i) * (ATS_KEYS + 1) + kk];
#pragma unroll
        for (int j = 0; j < DJ; ++j) vv[j] = Vs[kk * D + tc + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (pv[i] != 0.f) {
#pragma unroll
            for (int j = 0; j < DJ; ++j) o[i][j] = fmaf(pv[i], vv[j], o[i][j]);
          }
      }
    }
  }

  T* oh = out + ((size_t)(b * h_q + h) * C) * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + tr + 16 * i;
    if (t < C) {
      const float inv = 1.0f / l[i];          // every row sees at least its own key
#pragma unroll
      for (int j = 0; j < DJ; ++j) oh[(size_t)t * D + tc + 16 * j] = from_f32<T>(o[i][j] * inv);
    }
  }
}

}  // namespace quoka
