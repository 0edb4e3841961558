// Window attention on tensor cores (bf16): the chunk's queries over a sliding window of the
// contiguous cache and a few first tokens; out = softmax(q . k^T / sqrt(d)) . v over the keys
// j <= p with j < n_sink or j > p - window, p the query's position.
//
// A tile is a run of positions of one (sequence, KV head): 128 rows per SM pack the G query
// heads of the KV head at TP = 128 / G positions each.  d = 128 runs on SM pairs (clusters of
// two CTAs, 2 TP positions, 256-row tcgen05 MMAs with cta_group::2, each SM holding half of
// every K and V block), d = 64 on single SMs, whose K and V blocks are half the size.  K and V
// come straight from the cache by TMA: the keys of a tile are one run of rows after the first
// tokens, and blocks of 64 keys start at the oldest key that the tile's first position sees,
// so a tile walks the fewest blocks.  Tiles of neighbouring positions run at the same time and
// share most of their keys in L2.
//
// What bounds it is the softmax of the tiles: exponentials and products would each take 512
// clocks per block of 64 keys and SM, and windows make tiles short, so starting and finishing a
// tile weighs as much as ten blocks.  So every cluster runs two tiles at once, each with its own
// loader warp, MMA warp, four softmax warps, O in TMEM (columns 256 + 128 x), two buffers of S
// (columns 128 x and 128 x + 64, P over S), Q buffer and rings of four K and four V stages: one
// tile's start, end and masked blocks pass under the other's work.  S of block j + 2 is issued
// behind P.V of block j, so a softmax warp finds the next S done while its last block's products
// run.  A block then takes about 880 clocks per SM.  Measured on 4096 queries of 32 heads, 8 KV
// heads, window 4096, d 128: 257 us in a short run (1085 TFLOP/s; 265 without the exponentials on
// the FMA pipe below) and 296 among other calls, where the power limit lowers the clock.  8
// sequences of 1024 queries, 16 heads to a KV head, window 2047: 544 and 633 us.
// Steps of the design, each against what it replaced: two tiles at once 306, one tile whose blocks
// the two softmax groups share, as in attn_tc2.cuh, 320; blocks of 64 keys 266, blocks of 128, which
// leave TMEM for one S per tile, so that each tile's products and softmax wait for one another, 280
// (ragged 549, 616); a whole warp running the issuing loop 260, one thread, whose descriptors pass
// through general registers (70 clocks an MMA), 266.
// The clusters resident at once walk the tile list, cluster c taking tiles c, c + N, ...,
// its two streams in turn; the last of an odd number both streams share by key blocks, and
// stream 1's half reaches stream 0 through shared memory.
//
// Softmax: one thread per row of a tile, all 64 keys of a block.  The running maximum and sum
// are fp32; O is rescaled in TMEM only when the maximum grows by more than 2^8.  P is rounded to
// bf16 for its MMA (the row sum is taken from the unrounded weights).
//
// A block that not every row sees whole (the diagonal, the window's lower edge, the end of the
// first tokens) is masked by selection.  Its V tile is searched first for values that are not
// finite, in rows that nobody may see (another sequence's, or memory never written) or that
// some queries of the tile see: they are replaced by zero in shared memory and mark the tile,
// and the epilogue adds them to the rows that do see them.  Without this 0 * NaN would carry
// a masked row into every query of the tile.
//
// When the tiles are fewer than the clusters (short chunks), each tile's blocks are split over
// several units, which leave unnormalised partials (fp32) for the join kernel.
//
// Every mbarrier wait is bounded; the only unbounded waits are the block's and the cluster's
// barriers, which every thread reaches on every path.
#pragma once
#include <cooperative_groups.h>
#include <type_traits>
#include "attn_tc2.cuh"
#include "attn_window.cuh"

namespace quoka {

constexpr int AWT_THREADS = 384;   // warps 0-1 load, 2-3 MMA, 4-7 and 8-11 softmax
constexpr int AWT_ST = 4;          // K stages, and V stages, per stream
constexpr int AWT_BK = 64;         // keys per block
constexpr int AWT_FMA_EXP = 4;     // one of so many exponentials is taken on the FMA pipe: 257 us (3: 258, 5: 263, 8: 262, none 265)

template <int D>
struct AwtCfg {
  static constexpr bool PAIR = D == 128;
  static constexpr int CTAS = PAIR ? 2 : 1;        // CTAs per cluster
  static constexpr int KB = D / 64;
  static constexpr int Q_BYTES = 128 * D * 2;      // a CTA's query tile
  static constexpr int H_BYTES = 8192;             // a CTA's share of a K or V block
  static constexpr int STREAM = Q_BYTES + 2 * AWT_ST * H_BYTES;
  static constexpr int BARS = 5 + 5 * AWT_ST;      // per stream
  static constexpr int MBUF = 2 * 128 * 4;         // a shared unit's (m, l) of stream 1
  static constexpr int SMEM = 1024 + 2 * STREAM + (2 * BARS + 1) * 8 + 8 + 16 + 16 + MBUF;
};

// A unit of work: blocks [j0, j1) of the nblk blocks of a tile.
struct WindowUnit {
  int b, g, t0;
  int p_lo, p_hi;                  // absolute positions of the tile's first and last query
  int ns, w0, nsb;                 // first tokens [0, ns) in nsb blocks, then keys w0 .. p_hi
  int j0, j1;
  long long row0;                  // cache row of the sequence's position 0

  __device__ __forceinline__ int start(int j) const { return j < nsb ? j * AWT_BK : w0 + (j - nsb) * AWT_BK; }
  __device__ __forceinline__ int end(int j) const { return j < nsb ? ns : p_hi + 1; }
  // every query of the tile sees every key of block j
  __device__ __forceinline__ bool whole(int j, int window, int n_sink) const {
    const int k0 = start(j);
    return k0 + AWT_BK <= end(j) && k0 + AWT_BK - 1 <= p_lo && (k0 > p_hi - window || k0 + AWT_BK <= n_sink);
  }
};

__device__ __forceinline__ WindowUnit window_unit(const WindowParams& p, const SeqTable& tab, int unit, int ntp,
                                                  int span) {
  WindowUnit u;
  const unsigned tile = (unsigned)unit / (unsigned)p.nsplit, rest = tile / (unsigned)ntp;
  u.t0 = (ntp - 1 - (int)(tile - rest * ntp)) * span;      // longest key ranges first
  u.b = (int)(rest / (unsigned)p.h_kv);
  u.g = (int)rest - u.b * p.h_kv;
  const int P = tab.prefix[u.b];
  u.p_lo = P + u.t0;
  u.p_hi = P + min(p.C, u.t0 + span) - 1;
  const WindowSpan s = window_span(u.p_lo, u.p_hi, p.window, p.n_sink);
  u.ns = s.ns;
  u.w0 = s.w0;
  u.nsb = (s.ns + AWT_BK - 1) / AWT_BK;
  const int nblk = u.nsb + (s.p1 - s.w0) / AWT_BK + 1;
  const unsigned sp = (unsigned)unit - tile * p.nsplit;    // nblk <= 2^25 and nsplit <= 32
  u.j0 = (int)(nblk * sp / (unsigned)p.nsplit);
  u.j1 = (int)(nblk * (sp + 1) / (unsigned)p.nsplit);
  u.row0 = (long long)u.g * p.rows_per_head + tab.kv_off[u.b];
  return u;
}

// Whether a thread's share of a V tile of 8 KB in shared memory (thread tg of 128: the 16-byte
// vectors tg, tg + 128, ...) holds values that are not finite.
__device__ __forceinline__ bool window_bad_v(const uint4* v, int tg) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {            // an exponent of ones carries into the sign's place
    const uint4 x = v[i * 128 + tg];
    any |= ((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) |
           ((x.z & 0x7F807F80u) + 0x00800080u) | ((x.w & 0x7F807F80u) + 0x00800080u);
  }
  return (any & 0x80008000u) != 0;
}

// Replaces those values by zero in the warp's share of such a tile and writes `value` to `mark` (and
// to `far`, the other CTA's, unless that is 0).  Lane 0 may then arrive relaxed for the whole warp: its
// fence is ordered behind the other lanes' stores.  Out of line: within the softmax loop it costs every
// block, whether it runs or not (4096 queries, window 4096: 259 us against 252).
__device__ __noinline__ void window_clean_v(uint4* v, int tg, volatile int* mark, uint32_t far, int value) {
  for (int i = 0; i < 4; ++i) {
    uint32_t* w = reinterpret_cast<uint32_t*>(v + i * 128 + tg);
    for (int k = 0; k < 4; ++k) {
      if ((w[k] & 0x7F80u) == 0x7F80u) w[k] &= 0xFFFF0000u;
      if ((w[k] & 0x7F800000u) == 0x7F800000u) w[k] &= 0xFFFFu;
    }
  }
  *mark = value;
  if (far) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(far), "r"(value) : "memory");
  ptx::fence_proxy_async_smem();
  __syncwarp();
  __threadfence();
}

// Adds the values of 16 columns of V that window_clean_v took out of the unit's blocks to one
// row's output: an infinity or NaN times a positive weight is itself.
__device__ __noinline__ void window_add_bad(float* o, const __nv_bfloat16* v, const WindowUnit& u, int pos, int window,
                                            int n_sink, int D) {
  for (int j = u.j0; j < u.j1; ++j) {
    if (u.whole(j, window, n_sink)) continue;
    const int k0 = u.start(j), k1 = min(min(k0 + AWT_BK, u.end(j)), pos + 1);
    for (int kk = k0; kk < k1; ++kk) {
      if (!(kk < n_sink || kk > pos - window)) continue;
      for (int c = 0; c < 16; ++c) {
        const float x = __bfloat162float(v[(u.row0 + kk) * D + c]);
        if (!isfinite(x)) o[c] += x;
      }
    }
  }
}

// v[i] of lane l (l = lane % 4) becomes v[l] of lane i, within each four lanes.
__device__ __forceinline__ void window_transpose4(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & o) continue;
      uint4 send = up ? v[i] : v[i + o];
      send.x = __shfl_xor_sync(0xffffffffu, send.x, o);
      send.y = __shfl_xor_sync(0xffffffffu, send.y, o);
      send.z = __shfl_xor_sync(0xffffffffu, send.z, o);
      send.w = __shfl_xor_sync(0xffffffffu, send.w, o);
      if (up) v[i] = send; else v[i + o] = send;
    }
  }
}

// 2^t for t <= 16 on the FMA pipe: 2^round(t) from its exponent bits times a polynomial of degree 5
// in the rest (|rest| <= 1/2; fitted for the least relative error by Remez exchange: 7.5e-8, in
// fp32 2.2e-7 = 2^-22.1, which is what ex2.approx may be off by too, so that a weight does not
// depend on its key's place in the block).  Below 2^-126 it is zero; NaN stays NaN.
__device__ __forceinline__ float2 window_exp2(float2 t) {
  const float2 magic = make_float2(12583039.f, 12583039.f);      // 3 * 2^22 + 127: its low bits get n + 127
  t = make_float2(ptx::max_nan(t.x, -127.f), ptx::max_nan(t.y, -127.f));
  const float2 n = ptx::add2(t, magic);
  const float2 r = ptx::add2(n, make_float2(-magic.x, -magic.y));
  const float2 f = ptx::fma2(r, make_float2(-1.f, -1.f), t);
  float2 q = ptx::fma2(f, make_float2(1.32764725e-3f, 1.32764725e-3f), make_float2(9.67554096e-3f, 9.67554096e-3f));
  q = ptx::fma2(q, f, make_float2(0.0555071309f, 0.0555071309f));
  q = ptx::fma2(q, f, make_float2(0.240221202f, 0.240221202f));
  q = ptx::fma2(q, f, make_float2(0.693146944f, 0.693146944f));
  q = ptx::fma2(q, f, make_float2(1.00000012f, 1.00000012f));
  return ptx::mul2(q, make_float2(__int_as_float(__float_as_int(n.x) << 23), __int_as_float(__float_as_int(n.y) << 23)));
}

// The low n bits (n held to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int D>
__global__ void __cluster_dims__(D == 128 ? 2 : 1, 1, 1) __launch_bounds__(AWT_THREADS, 1)
window_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const __grid_constant__ SeqTable tab,
                 const __grid_constant__ WindowParams p, const __nv_bfloat16* __restrict__ v_cache,
                 __nv_bfloat16* __restrict__ out) {
  using Cfg = AwtCfg<D>;
  constexpr bool PAIR = Cfg::PAIR;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster.block_rank() : 0u;
  // this warp's stream, and that stream's memory
  const int x = warp < 4 ? (warp & 1) : (warp - 4) >> 2;
  uint8_t* sQ = smem + x * Cfg::STREAM;
  uint8_t* sK = sQ + Cfg::Q_BYTES;
  uint8_t* sV = sK + AWT_ST * Cfg::H_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 2 * Cfg::STREAM) + x * Cfg::BARS;
  uint64_t* qfull = bars;                  // this CTA's query tile landed
  uint64_t* qpeer = bars + 1;              // (CTA 0) CTA 1's query tile landed
  uint64_t* qempty = bars + 2;             // the S MMAs reading it are done (both CTAs)
  uint64_t* pready = bars + 3;             // [block parity], CTA 0: the pair's softmax warps of the stream wrote P
  // [stage], both CTAs: S of the block is done, and with it every MMA before; its K stage is
  // free then
  uint64_t* sfull = bars + 5;
  uint64_t* vempty = sfull + AWT_ST;       // [stage], both CTAs: P.V of the block is done
  uint64_t* kfull = vempty + AWT_ST;       // [stage], CTA 0: the K bytes of both CTAs
  uint64_t* vfull = kfull + AWT_ST;        // [stage], this CTA's V bytes
  uint64_t* vpeer = vfull + AWT_ST;        // [stage], CTA 0: CTA 1's V landed
  uint64_t* end_bars = reinterpret_cast<uint64_t*>(smem + 2 * Cfg::STREAM) + 2 * Cfg::BARS;
  uint64_t* merge = end_bars;              // stream 1's half of a shared unit lies in its rings
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(end_bars + 2);
  // [stream][unit parity] unit number + 1 when a value of one of its cleaned V blocks was not finite
  volatile int* mark = reinterpret_cast<volatile int*>(tmem_slot + 4) + x * 2;
  float* mbuf = reinterpret_cast<float*>(tmem_slot + 8);   // [m, l][row]
  // [column][row] of stream 1's O of a shared unit: over its K and V stages, which are done by then
  float* obuf = reinterpret_cast<float*>(smem + Cfg::STREAM + Cfg::Q_BYTES);

  const int span = (PAIR ? 2 : 1) * p.TP;  // positions of a tile
  const int ntp = (p.C + span - 1) / span;
  const int units = ntp * p.h_kv * tab.batch * p.nsplit;
  const int ncl = (int)gridDim.x / Cfg::CTAS, cid = (int)blockIdx.x / Cfg::CTAS;
  // units of this cluster, and of this stream of it (the same for both CTAs)
  const int cl_units = cid < units ? (units - 1 - cid) / ncl + 1 : 0;
  const int my_units = (cl_units + 1) >> 1;
  constexpr uint16_t kBoth = 0x3;
  // the streams take the cluster's units in turn, and share the blocks of the last of an odd number
  auto shared_unit = [&](int it) { return 2 * it + 1 == cl_units; };
  auto unit_of = [&](int it, int x) {
    const bool sh = shared_unit(it);
    WindowUnit u = window_unit(p, tab, cid + (2 * it + (sh ? 0 : x)) * ncl, ntp, span);
    const int mid = u.j0 + (u.j1 - u.j0 + 1) / 2;
    if (sh && x == 0) u.j1 = mid;
    if (sh && x == 1) u.j0 = mid;
    return u;
  };
  auto unit_at = [&](int it) { return unit_of(it, x); };
  auto commit = [&](uint64_t* bar) {
    if constexpr (PAIR) ptx::tc_commit_pair(bar, kBoth);
    else ptx::tc_commit(bar);
  };
  // waits on a barrier that the other CTA of the pair arrives on
  auto wait_pair = [&](uint64_t* bar, uint32_t parity) {
    if constexpr (PAIR) return ptx::mbar_wait_cluster_sleep(bar, parity);
    else return ptx::mbar_wait_sleep(bar, parity);
  };

  if (threadIdx.x < 64 && lane == 0) {     // warps 0 and 1: their streams' barriers
    mark[0] = mark[1] = 0;
    ptx::mbar_init(qfull, 1);
    ptx::mbar_init(qpeer, 1);
    ptx::mbar_init(qempty, 1);
    for (int s = 0; s < 2; ++s) ptx::mbar_init(&pready[s], 4 * Cfg::CTAS);
    for (int s = 0; s < 5 * AWT_ST; ++s) ptx::mbar_init(&sfull[s], 1);   // through vpeer
    if (x == 0) ptx::mbar_init(merge, 4);
    ptx::fence_mbar_init();
  }
  if (warp == 2) {
    if constexpr (PAIR) {
      ptx::tmem_alloc_pair(tmem_slot, 512);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(tmem_slot, 512);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster.sync();      // barriers and TMEM of both CTAs ready
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 2) {
    // ---------------- loads ----------------
    if (lane == 0) {
      ptx::prefetch_tmap(&qmap);
      ptx::prefetch_tmap(&kmap);
      ptx::prefetch_tmap(&vmap);
    }
    bool ok = true;
    int jg = 0, uq = 0;                    // blocks, and units with blocks, so far
    for (int it = 0; it < my_units && ok; ++it) {
      const WindowUnit u = unit_at(it);
      if (u.j0 == u.j1) continue;
      for (int j = u.j0; j < u.j1 && ok; ++j, ++jg) {
        const int st = jg % AWT_ST;
        const uint32_t free = ((uint32_t)(jg / AWT_ST) & 1u) ^ 1u;   // the stage's block jg - AWT_ST
        const int row = (int)u.row0 + u.start(j);
        if (lane == 0) {
          uint8_t* k_st = sK + st * Cfg::H_BYTES;
          ok = ptx::mbar_wait_sleep(&sfull[st], free);
          if (ok) {
            if constexpr (PAIR) {
              if (rank == 0) ptx::mbar_expect_tx(&kfull[st], 2u * Cfg::H_BYTES);
              const uint32_t fbar = ptx::mapa_shared(ptx::smem_u32(&kfull[st]), 0);
#pragma unroll
              for (int kb = 0; kb < 2; ++kb)
                ptx::tma_load_2d_pair(k_st + kb * 4096, &kmap, fbar, kb * 64, row + 32 * (int)rank);
            } else {
              ptx::mbar_expect_tx(&kfull[st], (uint32_t)Cfg::H_BYTES);
              ptx::tma_load_2d(k_st, &kmap, &kfull[st], 0, row);
            }
          }
        }
        if (j == u.j0) {
          // Q: 32 groups of 4 rows; row r is head r / TP, position t0 + rank * TP + r % TP (rows
          // past G * TP or C repeat a valid row; never stored)
          if (lane == 0 && ok) ok = ptx::mbar_wait_sleep(qempty, ((uint32_t)uq & 1u) ^ 1u);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (lane == 0) ptx::mbar_expect_tx(qfull, (uint32_t)Cfg::Q_BYTES);
          __syncwarp();
          const int r0 = lane * 4;
          int rows[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = r0 + k;
            int hl = r / p.TP, t = u.t0 + (int)rank * p.TP + r % p.TP;
            if (hl >= p.G || t >= p.C) { hl = 0; t = u.t0; }
            rows[k] = (u.b * p.h_q + u.g * p.G + hl) * p.C + t;
          }
#pragma unroll
          for (int kb = 0; kb < Cfg::KB; ++kb)
            ptx::tma_gather4(sQ + kb * 16384 + r0 * 128, &qmap, qfull, kb * 64, rows[0], rows[1], rows[2], rows[3]);
        }
        if (lane == 0 && ok) {
          ok = ptx::mbar_wait_sleep(&vempty[st], free);
          if (ok) {
            ptx::mbar_expect_tx(&vfull[st], (uint32_t)Cfg::H_BYTES);
            ptx::tma_load_2d(sV + st * Cfg::H_BYTES, &vmap, &vfull[st], 64 * (int)rank, row);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      ++uq;
    }
  } else if (warp < 4) {
    if (PAIR && rank == 1 && lane == 0) {
      // ---------------- CTA 1: tell CTA 0 when this CTA's query tiles and V blocks landed ----------------
      const uint32_t qpeer_c0 = ptx::mapa_shared(ptx::smem_u32(qpeer), 0);
      const uint32_t vpeer_c0 = ptx::mapa_shared(ptx::smem_u32(vpeer), 0);
      bool ok = true;
      int jg = 0, uq = 0;
      for (int it = 0; it < my_units && ok; ++it) {
        const WindowUnit u = unit_at(it);
        if (u.j0 == u.j1) continue;
        ok = ptx::mbar_wait_sleep(qfull, (uint32_t)uq & 1u);
        if (!ok) break;
        ptx::mbar_arrive_cluster(qpeer_c0);
        ++uq;
        for (int j = u.j0; j < u.j1 && ok; ++j, ++jg) {
          ok = ptx::mbar_wait_sleep(&vfull[jg % AWT_ST], (uint32_t)(jg / AWT_ST) & 1u);
          if (ok) ptx::mbar_arrive_cluster(vpeer_c0 + (uint32_t)(jg % AWT_ST) * 8u);
        }
      }
    }
    // ---------------- MMA issuer: one warp per stream (of CTA 0 for the pair) ----------------
    // The whole warp runs the loop and one elected lane issues: with everything uniform and the
    // stream a constant the descriptors stay in uniform registers.
    auto issue = [&](auto stream) {
      constexpr int x = decltype(stream)::value;
      uint8_t* sQ = smem + x * Cfg::STREAM;
      uint8_t* sK = sQ + Cfg::Q_BYTES;
      uint8_t* sV = sK + AWT_ST * Cfg::H_BYTES;
      uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + 2 * Cfg::STREAM) + x * Cfg::BARS;
      uint64_t *qpeer = qfull + 1, *qempty = qfull + 2, *pready = qfull + 3, *sfull = qfull + 5;
      uint64_t *vempty = sfull + AWT_ST, *kfull = vempty + AWT_ST, *vfull = kfull + AWT_ST, *vpeer = vfull + AWT_ST;
      const bool lead = ptx::elect_one();
      auto commit_lead = [&](uint64_t* bar) { if (lead) commit(bar); };
      const uint32_t idesc_s = ptx::idesc_bf16(PAIR ? 256 : 128, AWT_BK, false);
      const uint32_t idesc_o = ptx::idesc_bf16(PAIR ? 256 : 128, D, true);
      const uint64_t q_d = ptx::sdesc_sw128(ptx::smem_u32(sQ), 16, 1024);
      const uint64_t k_d = ptx::sdesc_sw128(ptx::smem_u32(sK), 16, 1024);
      const uint64_t v_d = ptx::sdesc_sw128(ptx::smem_u32(sV), 16384, 1024);
      const uint32_t q_lo = (uint32_t)q_d, q_hi = (uint32_t)(q_d >> 32);
      const uint32_t k_lo = (uint32_t)k_d, k_hi = (uint32_t)(k_d >> 32);
      const uint32_t v_lo = (uint32_t)v_d, v_hi = (uint32_t)(v_d >> 32);
      const uint32_t s_t = tmem + (uint32_t)(x * 128), o_t = tmem + 256u + (uint32_t)(x * 128);
      auto all = [](bool v) { return __all_sync(0xffffffffu, v) != 0; };
      auto s_mmas = [&](int jj) {
        const uint32_t b0 = k_lo + (uint32_t)((jj % AWT_ST) * (Cfg::H_BYTES >> 4));
        const uint32_t s_b = s_t + (uint32_t)((jj & 1) * AWT_BK);
#pragma unroll
        for (int kb = 0; kb < Cfg::KB; ++kb)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a = q_lo + (uint32_t)(kb * 1024 + k * 2);
            const uint32_t bb = b0 + (uint32_t)(kb * 256 + k * 2);
            if (!lead) continue;
            if constexpr (PAIR) ptx::mma_bf16_ss_pair(s_b, a, q_hi, bb, k_hi, idesc_s, (kb | k) ? 1u : 0u);
            else ptx::mma_bf16_ss_lh(s_b, a, q_hi, bb, k_hi, idesc_s, (kb | k) ? 1u : 0u);
          }
      };
      auto k_landed = [&](int jj) { return wait_pair(&kfull[jj % AWT_ST], (uint32_t)(jj / AWT_ST) & 1u); };
      auto v_landed = [&](int jj) {
        const uint32_t ph = (uint32_t)(jj / AWT_ST) & 1u;
        return ptx::mbar_wait_sleep(&vfull[jj % AWT_ST], ph) &&
               (!PAIR || ptx::mbar_wait_cluster_sleep(&vpeer[jj % AWT_ST], ph));
      };
      bool ok = true;
      int jg = 0, uq = 0;
      for (int it = 0; it < my_units && ok; ++it) {
        const WindowUnit u = unit_of(it, x);
        const int n = u.j1 - u.j0;
        if (n == 0) continue;
        ok = all(ptx::mbar_wait_sleep(qfull, (uint32_t)uq & 1u) &&
                 (!PAIR || ptx::mbar_wait_cluster_sleep(qpeer, (uint32_t)uq & 1u)));
        for (int j = 0; j < min(n, 2) && ok; ++j) {
          ok = all(k_landed(jg + j));
          if (!ok) break;
          ptx::tc_fence_after();
          s_mmas(jg + j);
          commit_lead(&sfull[(jg + j) % AWT_ST]);
        }
        if (!ok) break;
        if (n <= 2) commit_lead(qempty);
        // every wait of a block comes before its MMAs, which are issued back to back
        for (int j = 0; j < n && ok; ++j, ++jg) {
          const bool more = j + 2 < n;
          ok = all(v_landed(jg) && (!more || k_landed(jg + 2)) &&
                   wait_pair(&pready[jg & 1], (uint32_t)(jg >> 1) & 1u));
          if (!ok) break;
          ptx::tc_fence_after();
          // P: bf16 pairs in the first 32 columns of S
          const uint32_t b0 = v_lo + (uint32_t)((jg % AWT_ST) * (Cfg::H_BYTES >> 4));
#pragma unroll
          for (int k = 0; k < AWT_BK / 16; ++k) {
            const uint32_t a = s_t + (uint32_t)((jg & 1) * AWT_BK + k * 8);
            const uint32_t acc = (j > 0 || k > 0) ? 1u : 0u;
            if (!lead) continue;
            if constexpr (PAIR) ptx::mma_bf16_ts_pair(o_t, a, b0 + (uint32_t)(k * 128), v_hi, idesc_o, acc);
            else ptx::mma_bf16_ts_lh(o_t, a, b0 + (uint32_t)(k * 128), v_hi, idesc_o, acc);
          }
          commit_lead(&vempty[jg % AWT_ST]);
          if (more) {
            s_mmas(jg + 2);                // over P: after P.V has read it (issued in order)
            commit_lead(&sfull[(jg + 2) % AWT_ST]);
          }
          if (j + 3 == n) commit_lead(qempty);  // the unit's last S: its query buffer is free
        }
        ++uq;
      }
    };
    if (rank == 0) {
      if (warp == 2) issue(std::integral_constant<int, 0>{});
      else issue(std::integral_constant<int, 1>{});
    }
  } else {
    // ---------------- softmax: one thread per row ----------------
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;                      // row of the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr0 = tmem + lane_off + (uint32_t)(x * 128);
    const uint32_t o_addr = tmem + lane_off + 256u + (uint32_t)(x * 128);
    const uint32_t pready_c0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(pready), 0) : 0u;
    bool ok = true;
    int jg = 0;
    for (int it = 0; it < my_units && ok; ++it) {
      const WindowUnit u = unit_at(it);
      const int pos = u.p_lo + (int)rank * p.TP + r % p.TP; // this row's position
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = u.j0; j < u.j1; ++j, ++jg) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep<2>(&sfull[jg % AWT_ST], (uint32_t)(jg / AWT_ST) & 1u));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t s_addr = s_addr0 + (uint32_t)((jg & 1) * AWT_BK);
        float s[AWT_BK];
#pragma unroll
        for (int c = 0; c < AWT_BK; c += 32) {
          uint32_t w[32];
          ptx::tmem_ld32(s_addr + (uint32_t)c, w);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[c + i] = __uint_as_float(w[i]);
        }
        ptx::tmem_ld_wait();
        if (!u.whole(j, p.window, p.n_sink)) {
          const int k0 = u.start(j), kend = u.end(j);
          // bits of this row: below min(kend, pos + 1), and at pos - window + 1 or later or below
          // n_sink
          const int hi = min(kend, pos + 1) - k0, lo = pos - p.window + 1 - k0, sk = p.n_sink - k0;
#pragma unroll
          for (int c = 0; c < AWT_BK; c += 32) {
            const uint32_t w = low_bits(hi - c) & (~low_bits(lo - c) | low_bits(sk - c));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((w >> i) & 1u)) s[c + i] = -INFINITY;
          }
          // clean this CTA's share of the V tile before P.V reads it (the stream's 128 threads)
          ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&vfull[jg % AWT_ST], (uint32_t)(jg / AWT_ST) & 1u));
          if (!ok) break;
          uint4* v_st = reinterpret_cast<uint4*>(sV + (jg % AWT_ST) * Cfg::H_BYTES);
          if (__any_sync(0xffffffffu, window_bad_v(v_st, r))) {
            // (this CTA's columns are in the other's rows too)
            const uint32_t far = PAIR ? ptx::mapa_shared(ptx::smem_u32(const_cast<int*>(mark + (it & 1))), rank ^ 1u) : 0u;
            window_clean_v(v_st, r, mark + (it & 1), far, it + 1);
          }
        }
        float mx;
        {
          float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
          for (int c = 4; c < AWT_BK - 4; c += 8) {
            m0 = ptx::max3(m0, s[c], s[c + 1]);
            m1 = ptx::max3(m1, s[c + 2], s[c + 3]);
            m2 = ptx::max3(m2, s[c + 4], s[c + 5]);
            m3 = ptx::max3(m3, s[c + 6], s[c + 7]);
          }
          m0 = ptx::max3(m0, s[AWT_BK - 4], s[AWT_BK - 3]);
          m1 = ptx::max3(m1, s[AWT_BK - 2], s[AWT_BK - 1]);
          mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
        }
        const float m_cand = mx * p.scale_log2;
        const bool grow = m_cand > m_run + AT2_RESCALE_LOG2 || (m_run == -INFINITY && m_cand > -INFINITY);
        float alpha = 1.f;
        if (grow) {
          alpha = (m_run == -INFINITY) ? 0.f : ptx::ex2_approx(m_run - m_cand);
          m_run = m_cand;
          l_run *= alpha;
        }
        const float m_use = (m_run == -INFINITY) ? 0.f : m_run;
        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), minus_m2 = make_float2(-m_use, -m_use);
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < AWT_BK; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 t = ptx::fma2(make_float2(s[c + 2 * i], s[c + 2 * i + 1]), scale2, minus_m2);
            const float2 e = i % AWT_FMA_EXP == AWT_FMA_EXP - 1
                                 ? window_exp2(t)
                                 : make_float2(ptx::ex2_approx(t.x), ptx::ex2_approx(t.y));
            l2[i & 1] = ptx::add2(l2[i & 1], e);
            pk[i] = pack_bf16x2(e.x, e.y);
          }
          ptx::tmem_st16(s_addr + (uint32_t)(c / 2), pk);
        }
        l_run += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        if (j > u.j0 && __any_sync(0xffffffffu, grow)) {
          // O holds the unit's earlier blocks once the P.V of the one before is done (this block's
          // waits for this warp)
          ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep<2>(&vempty[(jg - 1) % AWT_ST],
                                                               (uint32_t)((jg - 1) / AWT_ST) & 1u));
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            uint32_t w[16];
            ptx::tmem_ld16(o_addr + (uint32_t)c, w);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
            ptx::tmem_st16(o_addr + (uint32_t)c, w);
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        // relaxed arrive: P and the rescaled O are TMEM stores already completed by
        // tcgen05.wait::st and ordered by the fence above; a release would stall the warp on
        // unrelated memory operations (the stores of the unit before)
        if (lane == 0) {
          if constexpr (PAIR) ptx::mbar_arrive_cluster_relaxed(pready_c0 + (uint32_t)(jg & 1) * 8u);
          else ptx::mbar_arrive(&pready[jg & 1]);
        }
      }
      // epilogue: O is final once the unit's last P.V has released its stage (that commit covers
      // every earlier MMA; the stage's next release needs this warp's next P)
      if (ok && u.j1 > u.j0)
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&vempty[(jg - 1) % AWT_ST], (uint32_t)((jg - 1) / AWT_ST) & 1u));
      if (!ok) break;
      const float l_row = l_run;
      const bool sh = shared_unit(it);
      const bool dirty = mark[it & 1] == it + 1;
      const int hl = r / p.TP;
      const int t = u.t0 + (int)rank * p.TP + r % p.TP;
      // output row of this thread, -1 for none
      const int orow = hl < p.G && t < p.C ? (u.b * p.h_q + u.g * p.G + hl) * p.C + t : -1;
      float l_all = l_row;
      ptx::tc_fence_after();
      if (sh) {
        // a shared unit: stream 1 leaves O, m and l, stream 0 joins them to its own
        float* ob = obuf + r;
        if (x == 1) {
          for (int c = 0; c < (u.j1 > u.j0 ? D : 0); c += 16) {
            uint32_t w[16];
            ptx::tmem_ld16(o_addr + (uint32_t)c, w);
            ptx::tmem_ld_wait();
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(w[i]);
            if (dirty && orow >= 0) window_add_bad(y, v_cache + c, u, pos, p.window, p.n_sink, D);
#pragma unroll
            for (int i = 0; i < 16; ++i) ob[(c + i) * 128] = y[i];
          }
          mbuf[r] = m_run;
          mbuf[128 + r] = l_row;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(merge);
          continue;                        // (the cluster's last unit)
        }
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(merge, 0));
        if (!ok) break;
        const float m1 = mbuf[r], l1 = mbuf[128 + r];
        const float M = l1 != 0.f ? (l_row != 0.f ? fmaxf(m_run, m1) : m1) : m_run;
        const float f0 = l_row != 0.f ? ptx::ex2_approx(m_run - M) : 0.f;
        const float f1 = l1 != 0.f ? ptx::ex2_approx(m1 - M) : 0.f;
        l_all = (l_row != 0.f ? l_row * f0 : 0.f) + (l1 != 0.f ? l1 * f1 : 0.f);
        m_run = M;
        for (int c = 0; c < (u.j1 > u.j0 ? D : 0); c += 16) {   // (stream 0 has blocks when stream 1 has)
          uint32_t w[16];
          ptx::tmem_ld16(o_addr + (uint32_t)c, w);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float a = f0 != 0.f ? __uint_as_float(w[i]) * f0 : 0.f;
            w[i] = __float_as_uint(f1 != 0.f ? fmaf(ob[(c + i) * 128], f1, a) : a);
          }
          ptx::tmem_st16(o_addr + (uint32_t)c, w);
        }
        ptx::tmem_st_wait();
      }
      {
        const bool split = p.nsplit > 1;
        // split units leave O and (m, l); others every row's O / l (each sees its own key)
        const float inv_l = split ? 1.f : 1.f / l_all;
        const size_t prow = ((size_t)(cid + (2 * it + (sh ? 0 : x)) * ncl) * Cfg::CTAS + rank) * 128 + r;
        if (split) {
          p.part_ml[prow * 2] = m_run;
          p.part_ml[prow * 2 + 1] = l_all;
        }
        if (u.j0 == u.j1) continue;        // (a unit without blocks: O is not set)
        uint32_t w[2][32];                 // the next 32 columns are on their way while these are stored
        ptx::tmem_ld32(o_addr, w[0]);
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          ptx::tmem_ld_wait();
          if (c + 32 < D) ptx::tmem_ld32(o_addr + (uint32_t)(c + 32), w[(c / 32 + 1) & 1]);
          uint4 w4[4];                     // 32 output columns as bf16
#pragma unroll
          for (int cc = 0; cc < 32; cc += 16) {
            float o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(w[(c / 32) & 1][cc + i]) * inv_l;
            if (dirty && orow >= 0) {
              float y[16];                 // (its address is taken here alone: o stays in registers)
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = o[i];
              window_add_bad(y, v_cache + c + cc, u, pos, p.window, p.n_sink, D);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = y[i];
            }
            if (split) {
              float4* d4 = reinterpret_cast<float4*>(p.part + prow * D + c + cc);
              if (orow >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) d4[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint4& y = w4[cc / 8 + i];
              y.x = pack_bf16x2(o[8 * i], o[8 * i + 1]);
              y.y = pack_bf16x2(o[8 * i + 2], o[8 * i + 3]);
              y.z = pack_bf16x2(o[8 * i + 4], o[8 * i + 5]);
              y.w = pack_bf16x2(o[8 * i + 6], o[8 * i + 7]);
            }
          }
          if (!split) {
            // four lanes exchange their rows' vectors, so that each store writes 64 bytes of a row
            window_transpose4(w4, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = __shfl_sync(0xffffffffu, orow, (lane & ~3) + i);
              if (row >= 0)
                reinterpret_cast<uint4*>(out + (size_t)row * D + c)[lane & 3] = w4[i];
            }
          }
        }
        ptx::tc_fence_before();
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster.sync();      // the pair's MMAs and loads are over on both SMs
  if (warp == 2) {
    __syncwarp();
    ptx::tc_fence_after();
    if constexpr (PAIR) ptx::tmem_dealloc_pair(tmem, 512);
    else ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace quoka
