// The streaming attention of attn_stream.cuh on tensor cores (bf16): one new token per
// sequence, paged or contiguous cache, the same split of the work, partials and join.
//
// A CTA holds the G query rows of a KV head (padded to N = 16, 32 or 64) against 128-key
// tiles, with both products turned so that the long sides fill the MMA's 128 rows:
//   S [128 keys x N]  = K_tile Q^T          (A = K tile, K-major; B = Q)
//   O^T [128 dims x N] += V_tile^T P^T      (A = V tile, MN-major; B = P^T from shared memory)
// (d = 64: rows 64-127 of O^T are computed over the K tile behind V and never read).  The
// kernel is bound by HBM: a tile is 64 KB (d = 128) and an SM's share of the bandwidth brings
// one in about 1.5 us, twice what the chain S -> softmax -> P.V takes.  So one tile is worked
// on at a time while TMA fills the ring's other stages; what counts is that the loads never
// pause, which the even split of the tiles and the stages ahead see to.
//
// Warp 0 loads: pages are copied box by box (a box is the largest power of two of rows that
// divides the page size, at most 128), only boxes with a visible key, and marks the boxes
// whose page was bad.  Warp 1 issues S, warp 6 P.V, warps 2-5 run the softmax, one thread per
// key: its N logits come with one TMEM load.  The running maximum is common to the tile's keys
// and only moves when some logit exceeds it by 2^8 (one barrier with an or-reduction tells);
// then O^T is rescaled in TMEM.  Row sums are kept per thread and added up at the end of a
// segment.  V rows of keys that are not visible are zeroed in shared memory, since 0 * NaN
// would reach the sum; masked logits are replaced by selection.
#pragma once
#include "tc_ptx.cuh"
#include "attn_stream.cuh"

namespace quoka {

constexpr int STC2_THREADS = 224;         // warp 0 load, 1 S, 2-5 softmax, 6 P.V
constexpr float STC2_RESCALE_LOG2 = 8.0f;

template <int D, int N>
struct Stc2Cfg {
  static constexpr int KB = D / 64;                 // 128-byte blocks per row
  static constexpr int T_BYTES = AST_TILE * D * 2;  // one K or V tile
  static constexpr int STAGE = 2 * T_BYTES;         // V, then K
  static constexpr int NST = (D == 128 ? 3 : 6) * (N == 64 ? 2 : 3) / 3;   // what fits beside Q and P
  static constexpr int QB = N == 16 ? 2 : 1;        // Q buffers
  static constexpr int Q_BYTES = N * D * 2;
  static constexpr int P_BYTES = N * AST_TILE * 2;
  static constexpr int TMEM = N == 16 ? 64 : N == 32 ? 128 : 256;   // S twice, O^T
  // kfull, vfull, empty per stage; qfull[2], qempty[2], sfull[2], pready[2], pfree[2]
  static constexpr int NBAR = 3 * NST + 10;
  static constexpr int FIXED = NST * STAGE + QB * Q_BYTES + 2 * P_BYTES + NBAR * 8 + 16 + NST * 4 + 4 * N * 4 * 2 + 64;
  static constexpr int smem(int batch) { return 1024 + FIXED + (2 * batch + 1) * 4; }
};

// Barrier among nthreads; true when any of them gives true.
__device__ __forceinline__ bool named_bar_or(int id, int nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

template <int D, int N, bool kPaged>
__global__ void __launch_bounds__(STC2_THREADS, 1)
attn_stream_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ StreamParams p,
                      const __grid_constant__ SeqTable tab, int box /* rows per TMA box */, __nv_bfloat16* __restrict__ out) {
  using Cfg = Stc2Cfg<D, N>;
  constexpr int KB = Cfg::KB, NST = Cfg::NST, QB = Cfg::QB;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
  uint8_t* sKV = smem;                              // stage s: V at s * STAGE, K behind it
  uint8_t* sQ = sKV + NST * Cfg::STAGE;
  uint8_t* sP = sQ + QB * Cfg::Q_BYTES;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(sP + 2 * Cfg::P_BYTES);
  uint64_t* vfull = kfull + NST;
  uint64_t* empty = vfull + NST;                    // P.V of the stage's tile is done
  uint64_t* qfull = empty + NST;                    // [Q buffer: segment % QB]
  uint64_t* qempty = qfull + 2;
  uint64_t* sfull = qempty + 2;                     // [tile parity] S is there
  uint64_t* pready = sfull + 2;                     // P is there (and S read)
  uint64_t* pfree = pready + 2;                     // P.V has read P
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pfree + 2);
  uint32_t* boxes = tmem_slot + 4;                  // [stage] bit i: box i of the tile was loaded
  float* wred = reinterpret_cast<float*>(boxes + ((NST + 3) & ~3));   // [4 warps][N]
  int* base = reinterpret_cast<int*>(wred + 2 * 4 * N);
  int* lens = base + p.batch + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&kmap);
    ptx::prefetch_tmap(&vmap);
    ptx::prefetch_tmap(&qmap);
    for (int s = 0; s < 3 * NST; ++s) ptx::mbar_init(&kfull[s], 1);   // through empty
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&qfull[s], 1);
      ptx::mbar_init(&qempty[s], 1);
      ptx::mbar_init(&sfull[s], 1);
      ptx::mbar_init(&pready[s], 4);
      ptx::mbar_init(&pfree[s], 1);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, Cfg::TMEM);
    ptx::tmem_relinquish();
  }
  for (int b = threadIdx.x; b < p.batch; b += STC2_THREADS) lens[b] = stream_len<kPaged>(p, tab, b);
  __syncthreads();
  stream_bases_of(p, lens, base);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int tiles = base[p.batch] * p.h_kv;
  const int ctas = min(p.ctas, tiles);
  const int c = blockIdx.x;
  const int x0 = c < ctas ? stream_start(c, ctas, tiles) : 0, x1 = c < ctas ? stream_start(c + 1, ctas, tiles) : 0;
  auto seg_at = [&](int x) { return stream_seg_of(p, lens, base, x, x1); };

  if (warp == 0) {
    // ---------------- loads ----------------
    const int nb = AST_TILE / box;                  // boxes per tile
    bool ok = true;
    int n = 0, sn = 0;                              // tiles, segments so far
    for (int x = x0; x < x1 && ok; ++sn) {
      const StreamSeg sg = seg_at(x);
      if (lane == 0) {
        const int qb = sn % QB;
        ok = ptx::mbar_wait_sleep(&qempty[qb], ((uint32_t)(sn / QB) & 1u) ^ 1u);
        if (ok) {
          ptx::mbar_expect_tx(&qfull[qb], (uint32_t)Cfg::Q_BYTES);
          for (int kb = 0; kb < KB; ++kb)
            ptx::tma_load_2d(sQ + qb * Cfg::Q_BYTES + kb * N * 128, &qmap, &qfull[qb], kb * 64,
                             sg.b * p.h_q + sg.g * p.G);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      for (int i = 0; i < sg.cnt && ok; ++i, ++n) {
        const int st = n % NST;
        // lane i < nb: the pool row of box i, and whether it is loaded
        const int k0 = sg.span.tile(sg.i0 + i) * AST_TILE + lane * box;
        bool on = lane < nb && k0 < sg.span.n && (k0 < sg.span.ns || k0 + box > sg.span.lo);
        int row = 0;
        if (on) {
          const long long rr = stream_row<kPaged>(p, tab, sg.b, sg.g, k0);
          on = rr >= 0;
          row = on ? (int)rr : 0;                   // pools and caches hold fewer than 2^31 rows
        }
        const uint32_t set = __ballot_sync(0xffffffffu, on);
        if (lane == 0) ok = ptx::mbar_wait_sleep(&empty[st], ((uint32_t)(n / NST) & 1u) ^ 1u);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t bytes = (uint32_t)(__popc(set) * box * D * 2);
          boxes[st] = set;
          ptx::mbar_expect_tx(&kfull[st], bytes);
          ptx::mbar_expect_tx(&vfull[st], bytes);
        }
        __syncwarp();
        uint8_t* sV = sKV + st * Cfg::STAGE;
        // K boxes first, then V: copy e is box e % nb, 128-byte block (e / nb) % KB, of K or V
        for (int e = lane; e < ((2 * KB * nb + 31) & ~31); e += 32) {
          const int bi = e % nb, kb = (e / nb) % KB;
          const bool isv = e >= KB * nb;
          const int r = __shfl_sync(0xffffffffu, row, bi);
          if (e < 2 * KB * nb && ((set >> bi) & 1u))
            ptx::tma_load_2d(sV + (isv ? 0 : Cfg::T_BYTES) + kb * 16384 + bi * box * 128, isv ? &vmap : &kmap,
                             isv ? &vfull[st] : &kfull[st], kb * 64, r);
        }
      }
      x += sg.cnt;
    }
  } else if (warp == 1) {
    // ---------------- S = K Q^T ----------------
    if (lane == 0) {
      const uint32_t idesc = ptx::idesc_bf16(128, N, false);
      bool ok = true;
      int n = 0, sn = 0;
      for (int x = x0; x < x1 && ok; ++sn) {
        const StreamSeg sg = seg_at(x);
        ok = ptx::mbar_wait_sleep(&qfull[sn % QB], (uint32_t)(sn / QB) & 1u);
        for (int i = 0; i < sg.cnt && ok; ++i, ++n) {
          const int st = n % NST, buf = n & 1;
          ok = ptx::mbar_wait_sleep(&kfull[st], (uint32_t)(n / NST) & 1u) &&
               ptx::mbar_wait_sleep(&pready[buf], ((uint32_t)(n >> 1) & 1u) ^ 1u);   // S(n - 2) was read
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            const uint32_t a0 = ptx::smem_u32(sKV + st * Cfg::STAGE + Cfg::T_BYTES + kb * 16384);
            const uint32_t b0 = ptx::smem_u32(sQ + (sn % QB) * Cfg::Q_BYTES + kb * N * 128);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              ptx::mma_bf16_ss(tmem + (uint32_t)(buf * N), ptx::sdesc_sw128(a0 + ks * 32, 16, 1024),
                               ptx::sdesc_sw128(b0 + ks * 32, 16, 1024), idesc, (kb | ks) ? 1u : 0u);
          }
          ptx::tc_commit(&sfull[buf]);
        }
        if (ok) ptx::tc_commit(&qempty[sn % QB]);
        x += sg.cnt;
      }
    }
  } else if (warp == 6) {
    // ---------------- O^T += V^T P^T ----------------
    if (lane == 0) {
      const uint32_t idesc = ptx::idesc_bf16(128, N, false) | (1u << 15);   // A is MN-major
      bool ok = true;
      int n = 0;
      for (int x = x0; x < x1 && ok;) {
        const StreamSeg sg = seg_at(x);
        for (int i = 0; i < sg.cnt && ok; ++i, ++n) {
          const int st = n % NST, buf = n & 1;
          ok = ptx::mbar_wait_sleep(&vfull[st], (uint32_t)(n / NST) & 1u) &&
               ptx::mbar_wait_sleep(&pready[buf], (uint32_t)(n >> 1) & 1u);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t a0 = ptx::smem_u32(sKV + st * Cfg::STAGE);
          const uint32_t b0 = ptx::smem_u32(sP + buf * Cfg::P_BYTES);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)                    // 16 keys per MMA
            ptx::mma_bf16_ss(tmem + 2 * N, ptx::sdesc_sw128(a0 + ks * 2048, 16384, 1024),
                             ptx::sdesc_sw128(b0 + (ks >> 2) * (N * 128) + (ks & 3) * 32, 16, 1024), idesc,
                             (i | ks) ? 1u : 0u);
          ptx::tc_commit(&empty[st]);
          ptx::tc_commit(&pfree[buf]);
        }
        x += sg.cnt;
      }
    }
  } else {
    // ---------------- softmax: thread = key of the tile, and dimension of O^T ----------------
    const int quarter = warp & 3;
    const int kk = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_addr = tmem + lane_off + 2 * N;
    // this key's place in P^T: 64-key block, then row r of 128 bytes, 16-byte chunks swizzled
    uint8_t* p_key = sP + (kk >> 6) * (N * 128) + (kk & 7) * 2;
    const int p_chunk = (kk & 63) >> 3;
    bool ok = true;
    int n = 0;
    // Every warp of the group reaches every barrier of every tile and segment: after a failed
    // (timed-out) wait it skips the work but not the barriers.
    for (int x = x0; x < x1;) {
      const StreamSeg sg = seg_at(x);
      float m[N], l[N];
#pragma unroll
      for (int r = 0; r < N; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
      for (int i = 0; i < sg.cnt; ++i, ++n) {
        const int st = n % NST, buf = n & 1;
        const int j = sg.span.tile(sg.i0 + i) * AST_TILE + kk;
        bool vis = false;
        float s[N];
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&sfull[buf], (uint32_t)(n >> 1) & 1u) &&
                                                 ptx::mbar_wait_sleep(&kfull[st], (uint32_t)(n / NST) & 1u));
        if (ok) {
          ptx::tc_fence_after();
#pragma unroll
          for (int r0 = 0; r0 < N; r0 += 16) {
            uint32_t w[16];
            ptx::tmem_ld16(tmem + lane_off + (uint32_t)(buf * N + r0), w);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r0 + r] = __uint_as_float(w[r]);
          }
          ptx::tmem_ld_wait();
          vis = sg.span.visible(j) && ((boxes[st] >> (kk / box)) & 1u);
        }
        bool up = false;
#pragma unroll
        for (int r = 0; r < N; ++r) {
          s[r] = vis ? s[r] * p.scale_log2 : -INFINITY;
          if (r < p.G) up = up || s[r] > m[r] + STC2_RESCALE_LOG2;   // (m = -inf: any visible key)
        }
        if (p.logits) {
          float* lg = p.logits + ((size_t)(x + i) * AST_TILE + kk) * p.G;
          if ((p.G & 3) == 0) {
#pragma unroll
            for (int r = 0; r < N; r += 4)
              if (r < p.G) *reinterpret_cast<float4*>(lg + r) = make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
          } else {
#pragma unroll
            for (int r = 0; r < N; ++r)
              if (r < p.G) lg[r] = s[r];
          }
        }
        if (named_bar_or(1, 128, up)) {
          // the tile's maxima, and O^T and the sums rescaled to them
#pragma unroll
          for (int r = 0; r < N; ++r) {
            if (r >= p.G) break;
            float v = s[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            if (lane == (r & 31)) wred[quarter * N + r] = v;
          }
          ptx::named_bar(2, 128);
          float al[N];
#pragma unroll
          for (int r = 0; r < N; ++r) {
            al[r] = 1.f;
            if (r >= p.G) continue;
            const float mn = fmaxf(fmaxf(fmaxf(wred[r], wred[N + r]), fmaxf(wred[2 * N + r], wred[3 * N + r])), m[r]);
            if (mn > m[r]) {
              al[r] = ptx::ex2_approx(m[r] - mn);           // m = -inf: 0
              m[r] = mn;
              l[r] *= al[r];
            }
          }
          if (i > 0 && ok) {
            // O^T holds the segment's earlier tiles once P.V of the last one is done
            ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&empty[(n - 1) % NST], (uint32_t)((n - 1) / NST) & 1u));
            if (ok) ptx::tc_fence_after();
#pragma unroll
            for (int r0 = 0; r0 < N; r0 += 16) {
              if (r0 >= p.G || !ok) break;
              uint32_t w[16];
              ptx::tmem_ld16(o_addr + (uint32_t)r0, w);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int r = 0; r < 16; ++r) w[r] = __float_as_uint(__uint_as_float(w[r]) * al[r0 + r]);
              ptx::tmem_st16(o_addr + (uint32_t)r0, w);
            }
            ptx::tmem_st_wait();
          }
          ptx::named_bar(2, 128);                           // wred is free again
        }
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&pfree[buf], ((uint32_t)(n >> 1) & 1u) ^ 1u));
        if (!ok) continue;
#pragma unroll
        for (int r = 0; r < N; ++r) {
          if (r >= p.G) break;
          // (a row whose keys so far are all masked has m = -inf and weights 0)
          const float pr = m[r] == -INFINITY ? 0.f : ptx::ex2_approx(s[r] - m[r]);
          l[r] += pr;
          *reinterpret_cast<__nv_bfloat16*>(p_key + buf * Cfg::P_BYTES + r * 128 + ((p_chunk ^ (r & 7)) << 4)) =
              __float2bfloat16_rn(pr);
        }
        if (!vis) {                                         // P.V must not meet what lies there
          (void)ptx::mbar_wait_sleep(&vfull[st], (uint32_t)(n / NST) & 1u);
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            uint4* v4 = reinterpret_cast<uint4*>(sKV + st * Cfg::STAGE + kb * 16384 + kk * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e) v4[e] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&pready[buf]);
      }

      // the segment's sums and O^T: out when the unit is whole, else a partial
#pragma unroll
      for (int r = 0; r < N; ++r) {
        if (r >= p.G) break;
        const float v = warp_sum(l[r]);
        if (lane == (r & 31)) wred[(4 + quarter) * N + r] = v;
      }
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&empty[(n - 1) % NST], (uint32_t)((n - 1) / NST) & 1u));
      ptx::named_bar(2, 128);
      if (ok) {
        ptx::tc_fence_after();
        const float* lw = wred + 4 * N;
        const int slot = 2 * c + (x == x0 ? 0 : 1);
#pragma unroll
        for (int r0 = 0; r0 < N; r0 += 16) {
          if (r0 >= p.G) break;
          uint32_t w[16];
          ptx::tmem_ld16(o_addr + (uint32_t)r0, w);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int ri = 0; ri < 16; ++ri) {
            const int r = r0 + ri;
            if (r >= p.G) break;
            const float L = (lw[r] + lw[N + r]) + (lw[2 * N + r] + lw[3 * N + r]);
            const float o = __uint_as_float(w[ri]);
            if (sg.whole) {
              if (kk < D)
                out[((size_t)sg.b * p.h_q + (size_t)sg.g * p.G + r) * D + kk] = __float2bfloat16_rn(L == 0.f ? 0.f : o / L);
              if (kk == 0 && p.logits) {
                p.unit_ml[((size_t)sg.unit * p.G + r) * 2] = m[r];
                p.unit_ml[((size_t)sg.unit * p.G + r) * 2 + 1] = L == 0.f ? 0.f : 1.f / L;
              }
            } else {
              if (kk < D) p.part[((size_t)slot * p.G + r) * D + kk] = o;
              if (kk == 0) {
                p.part_ml[((size_t)slot * p.G + r) * 2] = m[r];
                p.part_ml[((size_t)slot * p.G + r) * 2 + 1] = L;
              }
            }
          }
        }
        ptx::tc_fence_before();
      }
      ptx::named_bar(2, 128);                               // the sums are read
      x += sg.cnt;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Cfg::TMEM);
  }
}

}  // namespace quoka
