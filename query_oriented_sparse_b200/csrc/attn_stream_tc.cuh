// The streaming attention of attn_stream.cuh on tensor cores (bf16): one new token per
// sequence, paged or contiguous cache, the same split of the work, partials and join.
//
// A CTA holds the G query rows of a KV head (padded to N = 16, 32 or 64) against 128-key
// tiles, with both products turned so that the long sides fill the MMA's 128 rows:
//   S [128 keys x N]  = K_tile Q^T          (A = K tile, K-major; B = Q)
//   O^T [128 dims x N] += V_tile^T P^T      (A = V tile, MN-major; B = P^T from shared memory)
// (d = 64: rows 64-127 of O^T are computed over the K tile behind V and never read).  The
// kernel is bound by HBM: a tile is 64 KB (d = 128), and an SM's share of the bandwidth brings
// one in about 1.5 us.  What counts is that the loads never pause, which the even split of the
// tiles and the ring's stages see to, and that the chain S -> softmax -> P.V keeps up, which
// takes two softmax groups: for N = 16 they take the tiles in turn, each with its own maximum,
// sum and O^T, joined at the end of a segment; for more rows, where a tile's exponentials
// weigh more than its barriers, each takes half of the rows of every tile.
//
// Loads: pages are copied box by box (a box is the largest power of two of rows that divides the
// page size, at most 128; 32 rows of the contiguous cache), only boxes with a visible key, and
// boxes whose page is bad are left out and marked.  A paged box is one copy: the tensor map splits
// rows into groups of eight and their two 128-byte halves, so that the copy lays down whole
// swizzle atoms [group][half][8 rows].  Small copies are bound by their number, not their bytes:
// one copy for both halves of a 16-row page took the 32-sequence decode step (1.26 GB) from 275 to
// 217 us, and four loading warps instead of one 32 sequences of 8K to 16K tokens at d 64 from 206
// to 167 (pages of 16) and 327 to 225 (pages of 8); from pages of 32 rows on nothing of this
// shows (6.4 TB/s at d 128, 5.7 at d 64).
//
// The softmax runs with one thread per key: its logits come with one TMEM load.  The running
// maximum is common to the tile's keys and only moves when some logit exceeds it by 2^8 (one
// barrier with an or-reduction tells); then O^T is rescaled in TMEM.  Row sums are kept per
// thread and added up at the end of a segment.  V rows of keys that are not visible are zeroed
// in shared memory, since 0 * NaN would reach the sum; masked logits are replaced by
// selection.  P is rounded to bf16 for its MMA (the sums are taken before).
#pragma once
#include "tc_ptx.cuh"
#include <climits>
#include "attn_stream.cuh"

namespace quoka {

// Warps: 0 loads Q and K, 1 issues S, 2-9 softmax, 10 P.V; for N = 16, 11 loads K with warp 0, 12 and
// 13 V; for more rows, whose softmax needs the registers, 11 loads V.
constexpr float STC2_RESCALE_LOG2 = 8.0f;

template <int D, int N>
struct Stc2Cfg {
  static constexpr int LW = N == 16 ? 2 : 1;        // loading warps per operand
  static constexpr int THREADS = N == 16 ? 448 : 384;
  static constexpr int KB = D / 64;                 // 128-byte blocks per row
  static constexpr int T_BYTES = AST_TILE * D * 2;  // one K or V tile
  static constexpr int STAGE = 2 * T_BYTES;         // V, then K
  static constexpr int NST = (D == 128 ? 3 : 6) * (N == 64 ? 2 : 3) / 3;   // what fits beside Q and P
  static constexpr int QB = N == 16 ? 2 : 1;        // Q buffers
  static constexpr int Q_BYTES = N * D * 2;
  static constexpr int P_BYTES = N * AST_TILE * 2;
  static constexpr bool BYROW = N > 16;             // the softmax groups share rows, not tiles
  static constexpr int NR = BYROW ? N / 2 : N;      // rows per thread
  static constexpr int TMEM = N == 64 ? 256 : N == 32 ? 128 : 64;   // S twice, then O^T (one per group)
  static constexpr int OB = BYROW ? 0 : (N * 128 + 2 * N) * 4;      // one group's O^T, m and l of a segment
  // kfull, vfull, empty per stage; qfull[2], qempty[2], sfull[2], pready[2], pfree[2]
  static constexpr int NBAR = 3 * NST + 10;
  static constexpr int FIXED = NST * STAGE + QB * Q_BYTES + 2 * P_BYTES + NBAR * 8 + 16 + NST * 4 + 16 * NR * 4 + OB + 64;
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
__global__ void __launch_bounds__(Stc2Cfg<D, N>::THREADS, 1)
attn_stream_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ StreamParams p,
                      const __grid_constant__ SeqTable tab, int box /* rows per TMA box */, __nv_bfloat16* __restrict__ out) {
  using Cfg = Stc2Cfg<D, N>;
  constexpr int KB = Cfg::KB, NST = Cfg::NST, QB = Cfg::QB;
  // bytes between a tile's groups of eight rows, and between their 128-byte halves
  constexpr int GS = kPaged ? 1024 * KB : 1024, HS = kPaged ? 1024 : 16384;
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
  float* wred = reinterpret_cast<float*>(boxes + ((NST + 3) & ~3));   // [maxima, sums][8 warps][rows]
  float* obuf = wred + 16 * Cfg::NR;                   // [row][dimension], then m, l
  int* base = reinterpret_cast<int*>(obuf + Cfg::OB / 4);
  int* lens = base + p.batch + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::launch_dependents();               // the join's blocks may be placed as SMs fall free; they wait for this grid
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&kmap);
    ptx::prefetch_tmap(&vmap);
    ptx::prefetch_tmap(&qmap);
    for (int s = 0; s < 3 * NST; ++s) ptx::mbar_init(&kfull[s], 1);   // through empty
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&qfull[s], 1);
      ptx::mbar_init(&qempty[s], 1);
      ptx::mbar_init(&sfull[s], 1);
      ptx::mbar_init(&pready[s], Cfg::BYROW ? 8 : 4);
      ptx::mbar_init(&pfree[s], 1);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, Cfg::TMEM);
    ptx::tmem_relinquish();
  }
  for (int b = threadIdx.x; b < p.batch; b += Cfg::THREADS) lens[b] = stream_len<kPaged>(p, tab, b);
  __syncthreads();
  stream_bases_of(p, lens, base);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int c = blockIdx.x;
  int x0, x1;
  stream_share(p, base, c, &x0, &x1);
  auto seg_at = [&](int x) { return stream_seg_of(p, lens, base, x, x1); };

  constexpr int LW = Cfg::LW;
  if (warp == 0 || warp > 10) {
    // ---------------- loads: Q and K, V (two warps take an operand's copies in turn: one issues a
    // copy about every 60 ns) ----------------
    const bool isv = warp >= 10 + LW;
    const int share = LW == 2 && (warp == 11 || warp == 13);
    const bool lead = share == 0;                   // of the two: counts the tile's bytes
    // The rows of 32 boxes (one per lane, several tiles) are looked up at a time, a batch ahead
    // of their copies: a table entry comes from L2 or HBM.
    const int nb = AST_TILE / box, tb = 32 / nb;    // boxes per tile, tiles per batch
    int page = -1, off = 0;                         // next batch: this lane's page (contiguous: row), row in the pool
    auto look = [&](int xb) {
      page = -1;
      off = 0;
      const int x = xb + lane / nb;
      if (x >= x1) return;
      const StreamSeg sg = stream_seg_of(p, lens, base, x, x + 1);
      const int k0 = sg.span.tile(sg.i0) * AST_TILE + (lane % nb) * box;
      if (k0 >= sg.span.n || !(k0 < sg.span.ns || k0 + box > sg.span.lo)) return;
      if constexpr (kPaged) {
        const int pg = k0 / p.kv.page_size;
        off = sg.g * p.kv.page_size + k0 - pg * p.kv.page_size;
        page = __ldg(p.kv.block_table + (size_t)sg.b * p.kv.max_pages + pg);
        if (page < 0) page = INT_MIN;               // (an entry that is not a page: -1 is a box that is not wanted)
      } else {
        page = (int)stream_row<false>(p, tab, sg.b, sg.g, k0);
      }
    };
    bool ok = true;
    int n = 0, sn = 0;                              // tiles, segments so far
    int row = 0, bi0 = 0;                           // current batch: this lane's row; its tiles' first lane
    uint32_t set = 0;
    look(x0);
    for (int x = x0; x < x1 && ok; ++sn) {
      const StreamSeg sg = seg_at(x);
      if (lane == 0 && warp == 0) {
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
        if (n % tb == 0) {                          // the next batch
          bool on = page != -1;
          if (kPaged && on && (page < 0 || page >= p.kv.num_pages)) {
            if (warp == 0) flag_error(ERR_BAD_INDEX);
            on = false;
          }
          // pools and caches hold fewer than 2^31 rows
          row = on ? (kPaged ? page * (p.h_kv * p.kv.page_size) + off : page) : 0;
          set = __ballot_sync(0xffffffffu, on);
          look(x0 + n + tb);
        }
        bi0 = (n % tb) * nb;
        const uint32_t mine = (set >> bi0) & (nb == 32 ? ~0u : (1u << nb) - 1u);
        if (lane == 0) ok = ptx::mbar_wait_sleep(&empty[st], ((uint32_t)(n / NST) & 1u) ^ 1u);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        uint64_t* full = (isv ? vfull : kfull) + st;
        if (lane == 0 && lead) {
          if (!isv) boxes[st] = mine;
          ptx::mbar_expect_tx(full, (uint32_t)(__popc(mine) * box * D * 2));
        }
        __syncwarp();
        uint8_t* dst = sKV + st * Cfg::STAGE + (isv ? 0 : Cfg::T_BYTES);
        const CUtensorMap* map = isv ? &vmap : &kmap;
        const int e = LW * lane + share;
        if constexpr (kPaged) {                     // copy e: box e
          const int r = __shfl_sync(0xffffffffu, row, bi0 + e % nb);
          if (e < nb && ((mine >> e) & 1u))
            ptx::tma_load_4d(dst + e * box * D * 2, map, full, 0, 0, 0, r >> 3);
        } else {                                    // copy e: half e / nb of box e % nb
          const int bi = e % nb, kb = e / nb;
          const int r = __shfl_sync(0xffffffffu, row, bi0 + bi);
          if (kb < KB && ((mine >> bi) & 1u))
            ptx::tma_load_2d(dst + kb * 16384 + bi * box * 128, map, full, kb * 64, r);
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
            const uint32_t a0 = ptx::smem_u32(sKV + st * Cfg::STAGE + Cfg::T_BYTES + kb * HS);
            const uint32_t b0 = ptx::smem_u32(sQ + (sn % QB) * Cfg::Q_BYTES + kb * N * 128);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              ptx::mma_bf16_ss(tmem + (uint32_t)(buf * N), ptx::sdesc_sw128(a0 + ks * 32, 16, GS),
                               ptx::sdesc_sw128(b0 + ks * 32, 16, 1024), idesc, (kb | ks) ? 1u : 0u);
          }
          ptx::tc_commit(&sfull[buf]);
        }
        if (ok) ptx::tc_commit(&qempty[sn % QB]);
        x += sg.cnt;
      }
    }
  } else if (warp == 10) {
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
            ptx::mma_bf16_ss(tmem + (uint32_t)(2 * N + (Cfg::BYROW ? 0 : buf * N)),
                             ptx::sdesc_sw128(a0 + ks * 2 * GS, KB == 1 ? 16384 : HS, GS),
                             ptx::sdesc_sw128(b0 + (ks >> 2) * (N * 128) + (ks & 3) * 32, 16, 1024), idesc,
                             (i >= (Cfg::BYROW ? 1 : 2) || ks > 0) ? 1u : 0u);
          ptx::tc_commit(&empty[st]);
          ptx::tc_commit(&pfree[buf]);
        }
        x += sg.cnt;
      }
    }
  } else {
    // ---------------- softmax: thread = key of the tile, and dimension of O^T ----------------
    constexpr bool BYROW = Cfg::BYROW;
    constexpr int NR = Cfg::NR;
    const int grp = (warp - 2) >> 2;
    const int r_lo = BYROW ? grp * NR : 0;                  // this group's rows
    const int rows = min(NR, p.G - r_lo);                   // (may be <= 0)
    const int quarter = warp & 3;
    const int kk = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_addr = tmem + lane_off + (uint32_t)(2 * N + grp * NR);
    // this key's place in P^T: 64-key block, then row r of 128 bytes, 16-byte chunks swizzled
    uint8_t* p_key = sP + (kk >> 6) * (N * 128) + (kk & 7) * 2 + r_lo * 128;   // (r_lo is a multiple of 8)
    const int p_chunk = (kk & 63) >> 3;
    float* wmax = wred + grp * 4 * NR;
    float* wsum = wred + 8 * NR + grp * 4 * NR;
    const int bar_g = 1 + grp;                              // this group's barrier
    bool ok = true;
    int n = 0;
    // Every warp of the group reaches every barrier of every tile and segment: after a failed
    // (timed-out) wait it skips the work but not the barriers.
    for (int x = x0; x < x1;) {
      const StreamSeg sg = seg_at(x);
      float m[NR], l[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
      bool started = false;                                 // O^T holds earlier tiles of the segment
      uint32_t seen = 0;                                    // a box was loaded: the group's tiles had a visible key
      for (int i = 0; i < sg.cnt; ++i, ++n) {
        const int st = n % NST, buf = n & 1;
        if (!BYROW && buf != grp) continue;
        const uint32_t ph = (uint32_t)(n >> 1) & 1u;
        const int j = sg.span.tile(sg.i0 + i) * AST_TILE + kk;
        bool vis = false;
        float s[NR];
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&sfull[buf], ph) &&
                                                 ptx::mbar_wait_sleep(&kfull[st], (uint32_t)(n / NST) & 1u));
        if (ok) {
          ptx::tc_fence_after();
#pragma unroll
          for (int r0 = 0; r0 < NR; r0 += 16) {
            uint32_t w[16];
            ptx::tmem_ld16(tmem + lane_off + (uint32_t)(buf * N + r_lo + r0), w);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r0 + r] = __uint_as_float(w[r]);
          }
          const uint32_t there = boxes[st];
          seen |= there;
          vis = sg.span.visible(j) && ((there >> (kk / box)) & 1u);
          ptx::tmem_ld_wait();
        }
        bool up = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          s[r] = vis ? s[r] * p.scale_log2 : -INFINITY;
          if (r < rows) up = up || s[r] > m[r] + STC2_RESCALE_LOG2;   // (m = -inf: any visible key)
        }
        if (p.logits) {
          float* lg = p.logits + ((size_t)(x + i) * AST_TILE + kk) * p.G + r_lo;
          if ((p.G & 3) == 0) {
#pragma unroll
            for (int r = 0; r < NR; r += 4)
              if (r < rows) *reinterpret_cast<float4*>(lg + r) = make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
          } else {
#pragma unroll
            for (int r = 0; r < NR; ++r)
              if (r < rows) lg[r] = s[r];
          }
        }
        // P.V two tiles back (of this P buffer) is done; by tiles, it was this group's last one
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&pfree[buf], ph ^ 1u));
        if (named_bar_or(bar_g, 128, up)) {
          // the tile's maxima, and O^T and the sums rescaled to them
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            if (r >= rows) break;
            const float v = ptx::warp_max(s[r]);
            if (lane == (r & 31)) wmax[quarter * NR + r] = v;
          }
          ptx::named_bar(bar_g, 128);
          float al[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            al[r] = 1.f;
            if (r >= rows) continue;
            const float mn = fmaxf(fmaxf(fmaxf(wmax[r], wmax[NR + r]), fmaxf(wmax[2 * NR + r], wmax[3 * NR + r])), m[r]);
            if (mn > m[r]) {
              al[r] = ptx::ex2_approx(m[r] - mn);           // m = -inf: 0
              m[r] = mn;
              l[r] *= al[r];
            }
          }
          if (started && ok) {
            if constexpr (BYROW) {                          // P.V of the tile before
              ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&pfree[(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1u));
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int r0 = 0; r0 < NR; r0 += 16) {
              if (r0 >= rows || !ok) break;
              uint32_t w[16];
              ptx::tmem_ld16(o_addr + (uint32_t)r0, w);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int r = 0; r < 16; ++r) w[r] = __float_as_uint(__uint_as_float(w[r]) * al[r0 + r]);
              ptx::tmem_st16(o_addr + (uint32_t)r0, w);
            }
            ptx::tmem_st_wait();
          }
          ptx::named_bar(bar_g, 128);                       // wmax is free again
        }
        if (!ok) continue;
        started = true;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (r >= rows) break;
          // (m = -inf: the row's keys so far are masked, s = -inf, and weigh 0, or NaN, which stays)
          const float pr = ptx::ex2_approx(s[r] - (m[r] == -INFINITY ? 0.f : m[r]));
          l[r] += pr;
          *reinterpret_cast<__nv_bfloat16*>(p_key + buf * Cfg::P_BYTES + r * 128 + ((p_chunk ^ (r & 7)) << 4)) =
              __float2bfloat16_rn(pr);
        }
        if (!vis && (!BYROW || grp == 0)) {                 // P.V must not meet what lies there
          (void)ptx::mbar_wait_sleep(&vfull[st], (uint32_t)(n / NST) & 1u);
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            uint4* v4 = reinterpret_cast<uint4*>(sKV + st * Cfg::STAGE + (kk >> 3) * GS + kb * HS + (kk & 7) * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e) v4[e] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&pready[buf]);
      }

      // the segment's sums, and its last P.V of this group
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (r >= rows) break;
        const float v = warp_sum(l[r]);
        if (lane == (r & 31)) wsum[quarter * NR + r] = v;
      }
      if (ok && started) {
        const int nl = BYROW || ((n - 1) & 1) == grp ? n - 1 : n - 2;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleep(&pfree[nl & 1], (uint32_t)(nl >> 1) & 1u));
      }
      ptx::named_bar(bar_g, 128);
      ptx::tc_fence_after();
      // row r's sum (1 where visible keys weigh nothing: all their logits are -infinity)
      auto row_sum = [&](int r) {
        const float v = (wsum[r] + wsum[NR + r]) + (wsum[2 * NR + r] + wsum[3 * NR + r]);
        return seen && v == 0.f ? 1.f : v;
      };
      const int slot = 2 * c + (x == x0 ? 0 : 1);
      auto finish = [&](int r, float o, float M, float L) {  // row r_lo + r, dimension kk
        const int row = r_lo + r;
        if (sg.whole) {
          if (kk < D)
            out[((size_t)sg.b * p.h_q + (size_t)sg.g * p.G + row) * D + kk] = __float2bfloat16_rn(stream_result(o, M, L));
          if (kk == 0 && p.logits) {
            p.unit_ml[((size_t)sg.unit * p.G + row) * 2] = M;
            p.unit_ml[((size_t)sg.unit * p.G + row) * 2 + 1] = L == 0.f ? 0.f : 1.f / L;
          }
        } else {
          if (kk < D) p.part[((size_t)slot * p.G + row) * D + kk] = o;
          if (kk == 0) {
            p.part_ml[((size_t)slot * p.G + row) * 2] = M;
            p.part_ml[((size_t)slot * p.G + row) * 2 + 1] = L;
          }
        }
      };
#pragma unroll
      for (int r0 = 0; r0 < NR; r0 += 16) {
        if (r0 >= rows) break;
        uint32_t w[16];
        ptx::tmem_ld16(o_addr + (uint32_t)r0, w);
        ptx::tmem_ld_wait();
        if constexpr (BYROW) {
#pragma unroll
          for (int ri = 0; ri < 16; ++ri) {
            const int r = r0 + ri;
            if (r >= rows || !ok) break;
            finish(r, __uint_as_float(w[ri]), m[r], row_sum(r));
          }
        } else {
          // One group leaves its half of the segment's tiles, the other joins it to its own and
          // stores: the one that the next tile (n) is not for, since its next proxy fence waits
          // for the stores (1.2 us).
          float* ml = obuf + N * 128;
          if (grp == (n & 1)) {
#pragma unroll
            for (int r = 0; r < N; ++r) {
              if (r >= rows) break;
              obuf[r * 128 + kk] = __uint_as_float(w[r]);
              if (kk == 0) {
                ml[r] = m[r];
                ml[N + r] = ok ? row_sum(r) : 0.f;
              }
            }
          }
          ptx::named_bar(3, 256);
          if (grp != (n & 1)) {
#pragma unroll
            for (int r = 0; r < N; ++r) {
              if (r >= rows || !ok) break;
              const float l0 = row_sum(r), l1 = ml[N + r];
              const float M = l1 != 0.f ? (l0 != 0.f ? fmaxf(m[r], ml[r]) : ml[r]) : m[r];
              // a group without visible keys has l = 0 and an O^T that may not be set
              const bool none = M == -INFINITY;              // (of both, then: factors of 1 keep their sums)
              const float f0 = l0 == 0.f ? 0.f : none ? 1.f : ptx::ex2_approx(m[r] - M);
              const float f1 = l1 == 0.f ? 0.f : none ? 1.f : ptx::ex2_approx(ml[r] - M);
              const float o = (l0 != 0.f ? __uint_as_float(w[r]) * f0 : 0.f) + (l1 != 0.f ? obuf[r * 128 + kk] * f1 : 0.f);
              finish(r, o, M, (l0 != 0.f ? l0 * f0 : 0.f) + (l1 != 0.f ? l1 * f1 : 0.f));
            }
          }
        }
      }
      ptx::tc_fence_before();
      ptx::named_bar(3, 256);                               // the sums are read, and the half in obuf
      if (kPaged && p.own_record && ok)                     // (unit_ml and the logits are this CTA's own)
        for (int e = threadIdx.x - 64; e < sg.cnt * AST_TILE; e += 256)
          stream_record_key(p, sg, sg.span.tile(sg.i0 + e / AST_TILE) * AST_TILE + e % AST_TILE,
                            p.logits + ((size_t)x * AST_TILE + e) * p.G);
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
