// Host side of the window, paged-cache and eviction calls: validation, workspace layout
// and launches.  Part of quoka_abi.cu's translation unit (its checks and launch helpers
// are used here).
#pragma once

namespace {

// Runs an entry point's body; a C++ exception (host memory) becomes a status.
template <typename F>
quoka_status guarded(F body) {
  try {
    return body();
  } catch (const std::exception&) {
    return fail(QUOKA_ERR_CUDA, "host memory exhausted");
  }
}

struct PagedDims {
  Dims d;
  int page, num_pages, max_pages;
};

quoka_status check_paged(const quoka_paged_shape* s, PagedDims* p) {
  if (!s) return fail(QUOKA_ERR_INVALID_ARG, "shape is NULL");
  if (s->batch < 1) return fail(QUOKA_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", s->batch);
  if (s->batch > QUOKA_MAX_PAGED_BATCH)
    return fail(QUOKA_ERR_UNSUPPORTED, "batch %d exceeds QUOKA_MAX_PAGED_BATCH=%d", s->batch, QUOKA_MAX_PAGED_BATCH);
  const quoka_shape one = {1, s->h_q, s->h_kv, s->head_dim, 1, s->dtype};
  quoka_status st = check_shape(&one, &p->d);
  if (st != QUOKA_OK) return st;
  p->d.batch = s->batch;
  if (s->page_size < 8 || s->page_size % 8 != 0 || s->page_size > QUOKA_MAX_PAGE)
    return fail(QUOKA_ERR_UNSUPPORTED, "page_size %d not supported (a multiple of 8 up to %d)", s->page_size,
                QUOKA_MAX_PAGE);
  if (s->num_pages < 1 || s->max_pages < 1)
    return fail(QUOKA_ERR_INVALID_ARG, "num_pages=%d and max_pages=%d must be >= 1", s->num_pages, s->max_pages);
  if ((long long)s->num_pages * s->h_kv >= (1ll << 31) / s->page_size)
    return fail(QUOKA_ERR_UNSUPPORTED, "the pools have 2^31 rows or more");
  if ((long long)s->max_pages * s->page_size >= (1ll << 31) - 4096)
    return fail(QUOKA_ERR_UNSUPPORTED, "max_pages * page_size is 2^31 or more");
  p->page = s->page_size;
  p->num_pages = s->num_pages;
  p->max_pages = s->max_pages;
  return QUOKA_OK;
}

KvView paged_view(const PagedDims& p, const int32_t* seq_len, const int32_t* table, int max_pages, int max_len) {
  KvView kv;
  kv.seq_len = seq_len;
  kv.block_table = table;
  kv.max_pages = max_pages;
  kv.page_size = p.page;
  kv.num_pages = p.num_pages;
  kv.max_len = max_len;
  kv.rows_per_head = 0;
  return kv;
}

SeqTable empty_table() {
  SeqTable t;
  memset(&t, 0, sizeof(t));
  return t;
}

// ---- one new token per sequence: the streaming attention ---------------------------------
constexpr int STREAM_UNIT_TILES = 4;   // tiles of a sequence up to which a CTA takes a unit whole
constexpr int STREAM_MAX_CTAS = 592;   // CTAs of the streaming kernels at most (their partials' space)

struct StreamWs {
  size_t part, part_ml, unit_ml, logits, total;
  long long max_tiles;                 // bound on the tile list's length
  int max_unit_tiles, ctas;
};

// max_keys: bound on the keys a query sees.
StreamWs stream_ws(const Dims& d, long long max_keys, bool record) {
  StreamWs w;
  // two extra tiles: the last of the first tokens and the window's first may both be cut
  w.max_unit_tiles = (int)((std::max<long long>(max_keys, 1) + AST_TILE - 1) / AST_TILE) + 2;
  w.max_tiles = (long long)d.batch * d.h_kv * w.max_unit_tiles;
  w.ctas = (int)std::min<long long>(STREAM_MAX_CTAS, w.max_tiles);
  size_t off = 0;
  w.part = off;
  off = align_up(off + (size_t)2 * w.ctas * d.G * d.D * 4, 256);
  w.part_ml = off;
  off = align_up(off + (size_t)2 * w.ctas * d.G * 2 * 4, 256);
  w.unit_ml = off;
  off = align_up(off + (record ? (size_t)d.batch * d.h_q * 2 * 4 : 0), 256);
  w.logits = off;
  off = align_up(off + (record ? (size_t)w.max_tiles * AST_TILE * d.G * 4 : 0), 256);
  w.total = off;
  return w;
}

// Launches a kernel that may start before the one ahead of it on the stream has finished (it
// waits for it itself).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

template <typename T, int D, int R, bool kPaged>
cudaError_t launch_stream_simt(StreamParams& p, const SeqTable& tab, int max_ctas, const void* q, const void* k,
                               const void* v, void* out, cudaStream_t st) {
  const int smem = ast_smem_bytes<T, D, R>(p.batch);
  // as many CTAs as fit the SMs at once
  if (!p.by_unit) p.ctas = std::min(max_ctas, sm_count() * std::max(1, std::min(4, 230000 / (smem + 1024))));
  cudaError_t e = ensure_smem(attn_stream_kernel<T, D, R, kPaged>, smem);
  if (e != cudaSuccess) return e;
  attn_stream_kernel<T, D, R, kPaged><<<dim3(p.ctas, (p.G + R - 1) / R), AdcCfg<T, D>::THREADS, smem, st>>>(
      reinterpret_cast<const T*>(q), reinterpret_cast<const T*>(k), reinterpret_cast<const T*>(v), p, tab,
      reinterpret_cast<T*>(out));
  return cudaGetLastError();
}

// fp32: query heads of a group in rows of up to 16 per CTA.
template <typename T, int D, bool kPaged>
cudaError_t launch_stream_rows(StreamParams& p, const SeqTable& tab, int max_ctas, const void* q, const void* k,
                               const void* v, void* out, cudaStream_t st) {
  int r = 1;
  while (r < std::min(p.G, 16)) r *= 2;
  switch (r) {
    case 1: return launch_stream_simt<T, D, 1, kPaged>(p, tab, max_ctas, q, k, v, out, st);
    case 2: return launch_stream_simt<T, D, 2, kPaged>(p, tab, max_ctas, q, k, v, out, st);
    case 4: return launch_stream_simt<T, D, 4, kPaged>(p, tab, max_ctas, q, k, v, out, st);
    case 8: return launch_stream_simt<T, D, 8, kPaged>(p, tab, max_ctas, q, k, v, out, st);
    default: return launch_stream_simt<T, D, 16, kPaged>(p, tab, max_ctas, q, k, v, out, st);
  }
}

// Row-major [rows, cols] bf16 pool, rows a multiple of 8, as groups of eight rows and halves of
// 64 columns: a box is box_rows rows whole, laid down as [group][half][8 rows][128 bytes].
quoka_status make_map_groups(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows,
                             const char* what) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(QUOKA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[4] = {64, 8, cols / 64, rows / 8};
  const cuuint64_t strides[3] = {cols * 2, 128, cols * 16};
  const cuuint32_t box[4] = {64, 8, (cuuint32_t)(cols / 64), box_rows / 8};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(QUOKA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed: %d", what, (int)r);
  return QUOKA_OK;
}

// bf16: one CTA per SM (or per unit).
template <int D, int N, bool kPaged>
quoka_status launch_stream_tc(StreamParams& p, const SeqTable& tab, int max_ctas, const void* q, const void* k,
                              const void* v, void* out, cudaStream_t st) {
  if (!p.by_unit) p.ctas = std::min(max_ctas, sm_count());
  // Rows per copy: a power of two that divides the pages; over the contiguous cache 32, since the
  // first tokens and the window's ends leave most of their tiles' rows unread
  int box = kPaged ? AST_TILE : 32;
  uint64_t rows = (uint64_t)p.h_kv * p.kv.rows_per_head;
  if (kPaged) {
    while (p.kv.page_size % box) box /= 2;
    rows = (uint64_t)p.kv.num_pages * p.h_kv * p.kv.page_size;
  }
  CUtensorMap qmap, kmap, vmap;
  quoka_status s;
  if ((s = make_map_bf16(&qmap, q, (uint64_t)p.batch * p.h_q, D, 64, N, "q")) != QUOKA_OK) return s;
  if (kPaged) {
    if ((s = make_map_groups(&kmap, k, rows, D, box, "k_pages")) != QUOKA_OK) return s;
    if ((s = make_map_groups(&vmap, v, rows, D, box, "v_pages")) != QUOKA_OK) return s;
  } else {
    if ((s = make_map_bf16(&kmap, k, rows, D, 64, box, "k_cache")) != QUOKA_OK) return s;
    if ((s = make_map_bf16(&vmap, v, rows, D, 64, box, "v_cache")) != QUOKA_OK) return s;
  }
  const int smem = Stc2Cfg<D, N>::smem(p.batch);
  cudaError_t e = ensure_smem(attn_stream_tc_kernel<D, N, kPaged>, smem);
  if (e != cudaSuccess) return cuda_fail(e, "attn_stream_tc smem");
  attn_stream_tc_kernel<D, N, kPaged><<<p.ctas, Stc2Cfg<D, N>::THREADS, smem, st>>>(qmap, kmap, vmap, p, tab, box,
                                                                          reinterpret_cast<__nv_bfloat16*>(out));
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "attn_stream_tc launch");
  prof_mark(st, "attn_stream_tc_kernel");
  return QUOKA_OK;
}

template <typename T, int D, bool kPaged>
quoka_status launch_stream(const Dims& d, const SeqTable& tab, StreamParams p, const StreamWs& w, const void* q,
                           const void* k, const void* v, void* out, unsigned char* ws, cudaStream_t st) {
  p.batch = d.batch;
  p.h_q = d.h_q;
  p.h_kv = d.h_kv;
  p.G = d.G;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)D);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
  p.unit_ml = reinterpret_cast<float*>(ws + w.unit_ml);
  p.logits = p.record ? reinterpret_cast<float*>(ws + w.logits) : nullptr;
  // Sequences of up to STREAM_UNIT_TILES tiles: a (sequence, KV head) per CTA and one launch, while
  // these CTAs are no more than the SMs (512 sequences and heads of 300 keys: 44 us against 40)
  p.by_unit = w.max_unit_tiles - 2 <= STREAM_UNIT_TILES && d.batch * d.h_kv <= sm_count();
  if (p.by_unit) p.ctas = d.batch * d.h_kv;
  // (fp32 with more than 16 heads to a group splits them over CTAs: their sums meet in the kernel)
  p.own_record = p.record && p.by_unit && (sizeof(T) == 2 || d.G <= 16);
  cudaError_t e;
  if constexpr (sizeof(T) == 2) {
    const quoka_status s = d.G <= 16   ? launch_stream_tc<D, 16, kPaged>(p, tab, w.ctas, q, k, v, out, st)
                           : d.G <= 32 ? launch_stream_tc<D, 32, kPaged>(p, tab, w.ctas, q, k, v, out, st)
                                       : launch_stream_tc<D, 64, kPaged>(p, tab, w.ctas, q, k, v, out, st);
    if (s != QUOKA_OK) return s;
  } else {
    if ((e = launch_stream_rows<T, D, kPaged>(p, tab, w.ctas, q, k, v, out, st)) != cudaSuccess)
      return cuda_fail(e, "attn_stream launch");
    prof_mark(st, "attn_stream_kernel");
  }
  if (p.by_unit && (!p.record || p.own_record)) return QUOKA_OK;
  const int jblocks = (d.batch * d.h_q + ASJ_ROWS - 1) / ASJ_ROWS;
  if ((e = launch_dependent(attn_stream_join_kernel<T, D, kPaged>, jblocks, ASJ_ROWS * 32, (2 * d.batch + 1) * 4, st, p,
                            tab, reinterpret_cast<T*>(out))) != cudaSuccess)
    return cuda_fail(e, "attn_stream_join launch");
  prof_mark(st, "attn_stream_join_kernel");
  if (p.record) {
    const int grid = (int)std::min<long long>(w.max_tiles, (long long)sm_count() * 16);
    if ((e = launch_dependent(attn_stream_record_kernel, grid, AST_TILE, (2 * d.batch + 1) * 4, st, p, tab)) != cudaSuccess)
      return cuda_fail(e, "attn_stream_record launch");
    prof_mark(st, "attn_stream_record_kernel");
  }
  return QUOKA_OK;
}

template <bool kPaged>
quoka_status run_stream(const Dims& d, const SeqTable& tab, const StreamParams& p, const StreamWs& w, const void* q,
                        const void* k, const void* v, void* out, unsigned char* ws, cudaStream_t st) {
  if (d.dt == QUOKA_F32)
    return d.D == 64 ? launch_stream<float, 64, kPaged>(d, tab, p, w, q, k, v, out, ws, st)
                     : launch_stream<float, 128, kPaged>(d, tab, p, w, q, k, v, out, ws, st);
  return d.D == 64 ? launch_stream<__nv_bfloat16, 64, kPaged>(d, tab, p, w, q, k, v, out, ws, st)
                   : launch_stream<__nv_bfloat16, 128, kPaged>(d, tab, p, w, q, k, v, out, ws, st);
}

quoka_status check_ws(const void* workspace, size_t ws_bytes, size_t need) {
  if (need == 0) return QUOKA_OK;
  if (!workspace) return fail(QUOKA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (!aligned(workspace, 256)) return fail(QUOKA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return fail(QUOKA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, need);
  return QUOKA_OK;
}

// ---- window over the contiguous cache -----------------------------------------------------
StreamWs window_ws(const Dims& d, int max_prefix) { return stream_ws(d, (long long)max_prefix + 1, false); }

// Tiles of the chunk forms, units per tile and the space of their partials.  A tile holds
// (rows / G) positions: bf16 d 128 two CTAs of 128 rows, bf16 d 64 one, fp32 one of 64 rows.
constexpr int WINDOW_PAIRS = 74;              // bf16, d 128: clusters of two SMs, whose two streams share a unit
constexpr int WINDOW_SINGLES = 148;           // bf16, d 64; fp32
constexpr int WINDOW_MIN_BLOCKS = 8;          // 64-key blocks per unit at least
constexpr int WINDOW_MAX_SPLIT = 32;

struct WindowWs {
  long long tiles;
  int TP, nsplit;
  size_t part, part_ml, total;
};

WindowWs window_tile_ws(const Dims& d, int max_prefix, int window) {
  WindowWs w;
  const bool tc = d.dt == QUOKA_BF16, pair = tc && d.D == 128;
  const int ctas = pair ? 2 : 1, cta_rows = tc ? 128 : AWS_ROWS, keys = tc ? AWT_BK : AWS_KEYS;
  w.TP = cta_rows / d.G;
  const int span = ctas * w.TP;
  w.tiles = (long long)((d.C + span - 1) / span) * d.h_kv * d.batch;
  const long long blocks = (std::min<long long>(window, (long long)max_prefix + 1) + span + keys - 1) / keys;
  const long long room = (pair ? WINDOW_PAIRS : WINDOW_SINGLES) / w.tiles;
  w.nsplit = (int)std::max<long long>(1, std::min(std::min(room, blocks / WINDOW_MIN_BLOCKS), (long long)WINDOW_MAX_SPLIT));
  const size_t rows = w.nsplit > 1 ? (size_t)w.tiles * w.nsplit * ctas * cta_rows : 0;
  w.part = 0;
  w.part_ml = align_up(rows * d.D * 4, 256);
  w.total = align_up(w.part_ml + rows * 8, 256);
  return w;
}

WindowParams window_params(const Dims& d, long long rows, int window, int n_sink, unsigned char* ws, const WindowWs& w) {
  WindowParams p;
  p.h_q = d.h_q;
  p.h_kv = d.h_kv;
  p.G = d.G;
  p.C = d.C;
  p.TP = w.TP;
  p.window = window;
  p.n_sink = n_sink;
  p.nsplit = w.nsplit;
  p.rows_per_head = rows;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)d.D);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
  return p;
}

template <typename T, int D, int CTAS, int ROWS>
quoka_status launch_window_join(const Dims& d, const WindowParams& p, void* out, cudaStream_t st) {
  if (p.nsplit == 1) return QUOKA_OK;
  const long long total = (long long)d.batch * d.h_q * d.C * (D / 8);
  window_join_kernel<T, D, CTAS, ROWS><<<(unsigned)((total + AWJ_THREADS - 1) / AWJ_THREADS), AWJ_THREADS, 0, st>>>(
      p, total, reinterpret_cast<T*>(out));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "window_join launch");
  prof_mark(st, "window_join_kernel");
  return QUOKA_OK;
}

template <int D>
quoka_status launch_window_simt(const Dims& d, const SeqTable& tab, long long rows, const void* q, const void* k,
                                const void* v, int window, int n_sink, void* out, unsigned char* ws, const WindowWs& w,
                                cudaStream_t st) {
  const WindowParams p = window_params(d, rows, window, n_sink, ws, w);
  cudaError_t e;
  if ((e = ensure_smem(window_simt_kernel<D>, AwsCfg<D>::SMEM)) != cudaSuccess) return cuda_fail(e, "window smem");
  window_simt_kernel<D><<<(unsigned)(w.tiles * w.nsplit), AWS_THREADS, AwsCfg<D>::SMEM, st>>>(
      reinterpret_cast<const float*>(q), reinterpret_cast<const float*>(k), reinterpret_cast<const float*>(v), tab, p,
      reinterpret_cast<float*>(out));
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "window launch");
  prof_mark(st, "window_simt_kernel");
  return launch_window_join<float, D, 1, AWS_ROWS>(d, p, out, st);
}

// Clusters of the window kernel that fit on the device at once.
template <int D>
int window_resident(int smem) {
  if (D != 128) return sm_count();
  static std::mutex mu;
  static std::map<int, int> cache;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  auto it = cache.find(dev);
  if (it != cache.end()) return it->second;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * sm_count(), 1, 1);
  cfg.blockDim = dim3(AWT_THREADS, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, (const void*)window_tc_kernel<D>, &cfg) != cudaSuccess || n <= 0) {
    (void)cudaGetLastError();
    n = sm_count() / 2;
  }
  cache[dev] = n;
  return n;
}

template <int D>
quoka_status launch_window_tc(const Dims& d, const SeqTable& tab, long long rows, const void* q, const void* k,
                              const void* v, int window, int n_sink, void* out, unsigned char* ws, const WindowWs& w,
                              cudaStream_t st) {
  using Cfg = AwtCfg<D>;
  const WindowParams p = window_params(d, rows, window, n_sink, ws, w);
  CUtensorMap qmap, kmap, vmap;
  quoka_status s;
  const uint64_t kv_rows = (uint64_t)d.h_kv * rows;
  if ((s = make_map_bf16(&qmap, q, (uint64_t)d.batch * d.h_q * d.C, D, 64, 1, "q_chunk")) != QUOKA_OK) return s;
  if ((s = make_map_bf16(&kmap, k, kv_rows, D, 64, AWT_BK / Cfg::CTAS, "k_cache")) != QUOKA_OK) return s;
  if ((s = make_map_bf16(&vmap, v, kv_rows, D, 64, AWT_BK, "v_cache")) != QUOKA_OK) return s;
  const int smem = Cfg::SMEM;
  cudaError_t e;
  if ((e = ensure_smem(window_tc_kernel<D>, smem)) != cudaSuccess) return cuda_fail(e, "window_tc smem");
  const int ncl = (int)std::min<long long>(w.tiles * w.nsplit, window_resident<D>(smem));
  window_tc_kernel<D><<<Cfg::CTAS * ncl, AWT_THREADS, smem, st>>>(qmap, kmap, vmap, tab, p,
                                                                  reinterpret_cast<const __nv_bfloat16*>(v),
                                                                  reinterpret_cast<__nv_bfloat16*>(out));
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "window_tc launch");
  prof_mark(st, "window_tc_kernel");
  return launch_window_join<__nv_bfloat16, D, Cfg::CTAS, 128>(d, p, out, st);
}

}  // namespace

extern "C" {

size_t window_chunk_attn_workspace_size(const quoka_shape* shape, int max_prefix, int window) {
  Dims d;
  if (check_shape(shape, &d) != QUOKA_OK || max_prefix < 0 || window < 1) return 0;
  if (d.C == 1) return window_ws(d, max_prefix).total;
  return window_tile_ws(d, max_prefix, window).total;
}

quoka_status window_chunk_attn(const quoka_shape* shape, const void* q_chunk, const void* k_cache,
                               const void* v_cache, const int64_t* kv_off, const int32_t* prefix_len, int window,
                               int n_sink, void* out, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> quoka_status {
    Dims d;
    quoka_status s = check_shape(shape, &d);
    if (s != QUOKA_OK) return s;
    if (!q_chunk || !k_cache || !v_cache || !out)
      return fail(QUOKA_ERR_INVALID_ARG, "q_chunk, k_cache, v_cache and out must be non-NULL");
    if (!aligned(q_chunk, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
      return fail(QUOKA_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
    if (out == q_chunk || out == k_cache || out == v_cache)
      return fail(QUOKA_ERR_INVALID_ARG, "out must not alias an input");
    if (window < 1) return fail(QUOKA_ERR_INVALID_ARG, "window must be >= 1 (got %d)", window);
    if (n_sink < 0) return fail(QUOKA_ERR_INVALID_ARG, "n_sink must be >= 0 (got %d)", n_sink);
    const int32_t budget[QUOKA_MAX_BATCH] = {0};
    SeqTable tab;
    long long rows = 0;
    if ((s = build_table(d, kv_off, prefix_len, budget, 1, &tab, &rows)) != QUOKA_OK) return s;
    if ((long long)d.h_kv * rows >= (1ll << 31) - 65536)
      return fail(QUOKA_ERR_UNSUPPORTED, "the cache has 2^31 rows or more");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d.C == 1) {
      const StreamWs w = window_ws(d, tab.max_prefix);
      if ((s = check_ws(workspace, ws_bytes, w.total)) != QUOKA_OK) return s;
      StreamParams p;
      memset(&p, 0, sizeof(p));
      p.kv.rows_per_head = rows;
      p.kv.max_len = tab.max_prefix + 1;
      p.window = window;
      p.n_sink = n_sink;
      return run_stream<false>(d, tab, p, w, q_chunk, k_cache, v_cache, out,
                               reinterpret_cast<unsigned char*>(workspace), st);
    }
    const WindowWs w = window_tile_ws(d, tab.max_prefix, window);
    if (w.tiles * w.nsplit >= (1ll << 30)) return fail(QUOKA_ERR_UNSUPPORTED, "more than 2^30 query tiles");
    if ((s = check_ws(workspace, ws_bytes, w.total)) != QUOKA_OK) return s;
    auto* ws = reinterpret_cast<unsigned char*>(workspace);
    if (d.dt == QUOKA_F32)
      return d.D == 64 ? launch_window_simt<64>(d, tab, rows, q_chunk, k_cache, v_cache, window, n_sink, out, ws, w, st)
                       : launch_window_simt<128>(d, tab, rows, q_chunk, k_cache, v_cache, window, n_sink, out, ws, w, st);
    return d.D == 64 ? launch_window_tc<64>(d, tab, rows, q_chunk, k_cache, v_cache, window, n_sink, out, ws, w, st)
                     : launch_window_tc<128>(d, tab, rows, q_chunk, k_cache, v_cache, window, n_sink, out, ws, w, st);
  });
}

quoka_status paged_append(const quoka_paged_shape* shape, const void* k_new, const void* v_new, int n_new,
                          void* k_pages, void* v_pages, float* record, const int32_t* block_table,
                          const int32_t* start, const int32_t* count, void* stream) {
  return guarded([&]() -> quoka_status {
    PagedDims p;
    quoka_status s = check_paged(shape, &p);
    if (s != QUOKA_OK) return s;
    if (!k_new || !v_new || !k_pages || !v_pages || !block_table || !start)
      return fail(QUOKA_ERR_INVALID_ARG, "k_new, v_new, k_pages, v_pages, block_table and start must be non-NULL");
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
        !aligned(record, 16) || !aligned(block_table, 4) || !aligned(start, 4) || !aligned(count, 4))
      return fail(QUOKA_ERR_INVALID_ARG, "row pointers must be 16-byte aligned, tables 4-byte aligned");
    if (k_new == k_pages || k_new == v_pages || v_new == k_pages || v_new == v_pages || k_pages == v_pages)
      return fail(QUOKA_ERR_INVALID_ARG, "the new rows and the pools must not alias");
    if (n_new < 1) return fail(QUOKA_ERR_INVALID_ARG, "n_new must be >= 1 (got %d)", n_new);
    if (n_new > QUOKA_MAX_CHUNK)
      return fail(QUOKA_ERR_UNSUPPORTED, "n_new %d exceeds QUOKA_MAX_CHUNK=%d", n_new, QUOKA_MAX_CHUNK);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int vpr = p.d.D * p.d.esz / 16;
    const long long total = (long long)p.d.batch * p.d.h_kv * n_new * vpr;
    const int grid = (int)std::min<long long>((total + PAGED_THREADS - 1) / PAGED_THREADS, (long long)sm_count() * 16);
    paged_append_kernel<<<grid, PAGED_THREADS, 0, st>>>(
        reinterpret_cast<const uint4*>(k_new), reinterpret_cast<const uint4*>(v_new), reinterpret_cast<uint4*>(k_pages),
        reinterpret_cast<uint4*>(v_pages), record, paged_view(p, nullptr, block_table, p.max_pages, 0), start, count,
        p.d.h_kv, n_new, vpr, total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "paged_append launch");
    prof_mark(st, "paged_append_kernel");
    return QUOKA_OK;
  });
}

size_t paged_decode_attn_workspace_size(const quoka_paged_shape* shape, int max_len, int with_record) {
  PagedDims p;
  if (check_paged(shape, &p) != QUOKA_OK || max_len < 1 || (long long)max_len > (long long)p.max_pages * p.page) return 0;
  return stream_ws(p.d, max_len, with_record != 0).total;
}

quoka_status paged_decode_attn(const quoka_paged_shape* shape, const void* q, const void* k_pages,
                               const void* v_pages, const int32_t* block_table, const int32_t* seq_len, int max_len,
                               int window, int n_sink, float* record, void* out, void* workspace, size_t ws_bytes,
                               void* stream) {
  return guarded([&]() -> quoka_status {
    PagedDims p;
    quoka_status s = check_paged(shape, &p);
    if (s != QUOKA_OK) return s;
    if (!q || !k_pages || !v_pages || !block_table || !seq_len || !out)
      return fail(QUOKA_ERR_INVALID_ARG, "q, k_pages, v_pages, block_table, seq_len and out must be non-NULL");
    if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(record, 16) ||
        !aligned(block_table, 4) || !aligned(seq_len, 4))
      return fail(QUOKA_ERR_INVALID_ARG, "row pointers must be 16-byte aligned, tables 4-byte aligned");
    if (out == q || out == k_pages || out == v_pages || out == (const void*)record)
      return fail(QUOKA_ERR_INVALID_ARG, "out must not alias an input");
    if (max_len < 1 || (long long)max_len > (long long)p.max_pages * p.page)
      return fail(QUOKA_ERR_INVALID_ARG, "max_len %d outside [1, max_pages * page_size = %lld]", max_len,
                  (long long)p.max_pages * p.page);
    if (window < 1) return fail(QUOKA_ERR_INVALID_ARG, "window must be >= 1 (got %d)", window);
    if (n_sink < 0) return fail(QUOKA_ERR_INVALID_ARG, "n_sink must be >= 0 (got %d)", n_sink);
    const StreamWs w = stream_ws(p.d, max_len, record != nullptr);
    if (w.max_tiles >= (1ll << 31)) return fail(QUOKA_ERR_UNSUPPORTED, "more than 2^31 key tiles");
    if ((s = check_ws(workspace, ws_bytes, w.total)) != QUOKA_OK) return s;
    StreamParams sp;
    memset(&sp, 0, sizeof(sp));
    sp.kv = paged_view(p, seq_len, block_table, p.max_pages, max_len);
    sp.window = window;
    sp.n_sink = n_sink;
    sp.record = record;
    return run_stream<true>(p.d, empty_table(), sp, w, q, k_pages, v_pages, out,
                            reinterpret_cast<unsigned char*>(workspace), reinterpret_cast<cudaStream_t>(stream));
  });
}

quoka_status paged_evict(const quoka_paged_shape* shape, void* k_pages, void* v_pages, float* record,
                         const int32_t* block_table, const int32_t* seq_len, int max_len, const int32_t* budget,
                         int b_max, int n_sink, int n_recent, const int32_t* dst_table, int dst_max_pages,
                         int32_t* idx_out, int32_t* new_len, void* stream) {
  return guarded([&]() -> quoka_status {
    PagedDims p;
    quoka_status s = check_paged(shape, &p);
    if (s != QUOKA_OK) return s;
    if (!k_pages || !v_pages || !record || !block_table || !seq_len || !budget || !dst_table || !idx_out || !new_len)
      return fail(QUOKA_ERR_INVALID_ARG, "a pool, table, length or output is NULL");
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(record, 16) || !aligned(block_table, 4) ||
        !aligned(seq_len, 4) || !aligned(budget, 4) || !aligned(dst_table, 4) || !aligned(idx_out, 16) ||
        !aligned(new_len, 4))
      return fail(QUOKA_ERR_INVALID_ARG, "row pointers must be 16-byte aligned, tables 4-byte aligned");
    if (k_pages == v_pages || dst_table == block_table || new_len == seq_len || new_len == budget)
      return fail(QUOKA_ERR_INVALID_ARG, "the pools must differ, and outputs must not alias inputs");
    if (max_len < 1 || (long long)max_len > (long long)p.max_pages * p.page)
      return fail(QUOKA_ERR_INVALID_ARG, "max_len %d outside [1, max_pages * page_size = %lld]", max_len,
                  (long long)p.max_pages * p.page);
    if (max_len > QUOKA_MAX_EVICT_LEN)
      return fail(QUOKA_ERR_UNSUPPORTED, "max_len %d exceeds QUOKA_MAX_EVICT_LEN=%d", max_len, QUOKA_MAX_EVICT_LEN);
    if (dst_max_pages < 1 || b_max < 1 || (long long)b_max > (long long)dst_max_pages * p.page)
      return fail(QUOKA_ERR_INVALID_ARG, "b_max %d outside [1, dst_max_pages * page_size = %lld]", b_max,
                  (long long)dst_max_pages * p.page);
    if (n_sink < 0 || n_recent < 0)
      return fail(QUOKA_ERR_INVALID_ARG, "n_sink=%d and n_recent=%d must be >= 0", n_sink, n_recent);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const KvView kv = paged_view(p, seq_len, block_table, p.max_pages, max_len);
    const KvView dst = paged_view(p, nullptr, dst_table, dst_max_pages, 0);
    const int nrows = p.d.batch * p.d.h_kv;
    // CTAs per row: 16, halved while the rows' clusters would not all fit the SMs at once
    // and a CTA's slice still fits its staging area
    int cs = EVS_MAX_CS;
    while (cs > 1 && (long long)nrows * cs > (long long)sm_count() && (max_len + cs / 2 - 1) / (cs / 2) <= EVS_STAGE_KEYS)
      cs /= 2;
    // slices so long that a CTA fills an SM: more and shorter ones, while they fit the SMs together
    while (cs < EVS_MAX_CS && (max_len + cs - 1) / cs > EVS_SHARE_KEYS && (long long)nrows * cs * 2 <= 4LL * sm_count()) cs *= 2;
    const int smem = std::max((max_len + cs - 1) / cs, 1) * 4;
    auto launch = [&](auto kern, int csz) -> cudaError_t {
      cudaError_t err = ensure_smem(kern, smem);
      if (err == cudaSuccess && csz > 8) err = ensure_cluster16(kern);
      if (err != cudaSuccess) return err;
      kern<<<nrows * csz, EVS_THREADS, smem, st>>>(record, kv, budget, p.d.h_kv, b_max, n_sink, n_recent, idx_out, new_len);
      return cudaGetLastError();
    };
    cudaError_t e;
    switch (cs) {
      case 1: e = launch(evict_select_kernel<1>, 1); break;
      case 2: e = launch(evict_select_kernel<2>, 2); break;
      case 4: e = launch(evict_select_kernel<4>, 4); break;
      case 8: e = launch(evict_select_kernel<8>, 8); break;
      default: e = launch(evict_select_kernel<16>, 16); break;
    }
    if (e != cudaSuccess) return cuda_fail(e, "evict_select launch");
    prof_mark(st, "evict_select_kernel");
    const dim3 cgrid(nrows, (std::min(b_max, max_len) + EVC_WARPS * 32 - 1) / (EVC_WARPS * 32));
    auto copy = [&](auto kern) {
      return launch_dependent(kern, cgrid, EVC_WARPS * 32, 0, st, reinterpret_cast<uint4*>(k_pages),
                              reinterpret_cast<uint4*>(v_pages), record, kv, dst, idx_out, new_len, p.d.h_kv, b_max);
    };
    switch (p.d.D * p.d.esz / 16) {
      case 8: e = copy(evict_copy_kernel<8>); break;
      case 16: e = copy(evict_copy_kernel<16>); break;
      default: e = copy(evict_copy_kernel<32>); break;
    }
    if (e != cudaSuccess) return cuda_fail(e, "evict_copy launch");
    prof_mark(st, "evict_copy_kernel");
    return QUOKA_OK;
  });
}

}  // extern "C"
