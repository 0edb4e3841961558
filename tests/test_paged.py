"""The paged cache: append, one-token attention over pages with and without a weight record,
eviction by that record, and the three together, against the plain 64-bit forms."""
import ctypes

import pytest
import torch

import bounded_ref as R
from query_oriented_sparse_b200 import binding as Bd

BF, F32 = torch.bfloat16, torch.float32


class Pool:
    """Pools on the CPU whose unused slots hold NaN, with shuffled pages."""

    def __init__(self, h_kv, d, page, lens, dtype, seed=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        per = [-(-n // page) for n in lens]
        N = sum(per) + spare
        perm = torch.randperm(N, generator=g).tolist()
        self.page, self.lens = page, list(lens)
        self.table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32)
        self.k = torch.full((N, h_kv, page, d), float("nan"), dtype=dtype)
        self.v = torch.full((N, h_kv, page, d), float("nan"), dtype=dtype)
        self.w = torch.full((N, h_kv, page), float("nan"))
        for b, (n, m) in enumerate(zip(lens, per)):
            pages = [perm.pop() for _ in range(m)]
            self.table[b, :m] = torch.tensor(pages, dtype=torch.int32)
            for i, p in enumerate(pages):
                r = min(page, n - i * page)
                self.k[p, :, :r] = torch.randn(h_kv, r, d, generator=g).to(dtype)
                self.v[p, :, :r] = torch.randn(h_kv, r, d, generator=g).to(dtype)
                self.w[p, :, :r] = torch.rand(h_kv, r, generator=g)
        self.free = perm
        self.seq_len = torch.tensor(lens, dtype=torch.int32)

    def gpu(self):
        return self.k.cuda(), self.v.cuda(), self.table.cuda(), self.seq_len.cuda()


def decode_ref(pool, q, window, n_sink):
    """Per sequence and KV head: out, tolerance, weights summed over the group, their bound."""
    B, h_q, _, d = q.shape
    h_kv = pool.k.shape[1]
    G = h_q // h_kv
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    w, we = [], []
    for b, n in enumerate(pool.lens):
        j = torch.arange(n)
        seen = ((j < n_sink) | (j >= n - window)).expand(G, n)
        ks, vs = R.gather_pages(pool.k, pool.table[b], n), R.gather_pages(pool.v, pool.table[b], n)
        wb, eb = torch.zeros(h_kv, n, dtype=torch.float64), torch.zeros(h_kv, n, dtype=torch.float64)
        for g in range(h_kv):
            kk = torch.where(seen[0][:, None], ks[g].double(), 0.0)
            vv = torch.where(seen[0][:, None], vs[g].double(), 0.0)
            o, mag, p, S = R.attend(q[b, g * G:(g + 1) * G, 0].double(), kk, vv, seen)
            nn = seen.sum(-1, keepdim=True)
            out[b, g * G:(g + 1) * G, 0] = o
            tol[b, g * G:(g + 1) * G, 0] = R.out_tol(o, mag, S, d, nn, q.dtype)
            wb[g] = p.sum(0)
            eb[g] = (p * R.weight_err(d, nn, S)).sum(0) + G * 2.0 ** -24 * p.sum(0)
        w.append(wb)
        we.append(eb)
    return out, tol, w, we


LENS = [(0, 1, 7, 8, 9), (127, 128, 129, 0), (1000, 3), (5000,), tuple(range(40, 360, 4))]
SHAPES = [(4, 1, 64), (4, 1, 128), (8, 8, 128), (10, 2, 128), (16, 1, 64), (48, 2, 128), (64, 1, 128), (64, 1, 64)]


def run_decode(pool, q, window=None, n_sink=0, record=False, max_len=None):
    k, v, table, lens = pool.gpu()
    w = pool.w.cuda() if record else None
    out = torch.full_like(q, float("nan")).cuda()
    Bd.paged_decode_attn(q.cuda(), k, v, table, lens, max_len or max(max(pool.lens), 1), window=window, n_sink=n_sink,
                         weight_pages=w, out=out)
    return out.cpu(), None if w is None else w.cpu()


def check_decode(pool, q, window, n_sink, out, w):
    big = max(max(pool.lens), 1)
    ref, tol, rw, we = decode_ref(pool, q, window or big, n_sink)
    R.assert_close(out, ref, tol, "out")
    if w is None:
        return
    touched = torch.zeros_like(w, dtype=torch.bool)
    for b, n in enumerate(pool.lens):
        if n == 0:
            continue
        was = R.gather_pages(pool.w, pool.table[b], n).double()
        got = R.gather_pages(w, pool.table[b], n).double()
        want = was + rw[b]
        R.assert_close(got, want, we[b] + want.abs() * 2.0 ** -24, f"record of sequence {b}")
        j = torch.arange(n)
        touched[pool.table[b][j // pool.page].long(), :, j % pool.page] = True
    assert torch.equal(w[~touched].isnan(), pool.w[~touched].isnan())   # the other slots are as they were


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("page", [8, 16, 24, 64, 128, 256, 1024])
@pytest.mark.parametrize("i", range(len(LENS)))
def test_decode_lengths_and_pages(i, page, dtype, cuda_device):
    h_q, h_kv, d = SHAPES[(i + page // 8) % len(SHAPES)]
    pool = Pool(h_kv, d, page, LENS[i], dtype, seed=i)
    q = (1.5 * torch.randn(len(LENS[i]), h_q, 1, d, generator=torch.Generator().manual_seed(i))).to(dtype)
    out, w = run_decode(pool, q, record=True)
    assert Bd.device_error() == 0
    check_decode(pool, q, None, 0, out, w)
    out2, _ = run_decode(pool, q, max_len=pool.table.shape[1] * page)   # a looser bound, no record
    R.assert_close(out2, *decode_ref(pool, q, 1 << 30, 0)[:2], "out without a record")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("window,n_sink", [(1, 0), (100, 4), (128, 128), (300, 200), (700, 1), (5, 100000), (100000, 0)])
def test_decode_window(window, n_sink, shape, dtype, cuda_device):
    h_q, h_kv, d = shape
    pool = Pool(h_kv, d, 16, (1000, 130, 5, 0), dtype, seed=7)
    # pages that no query sees have been given back: their entries are -1
    full = pool.table.clone()
    for b, n in enumerate(pool.lens):
        for p in range(-(-n // 16)):
            if p * 16 >= n_sink and p * 16 + 16 <= n - window:
                pool.table[b, p] = -1
    q = (1.5 * torch.randn(4, h_q, 1, d, generator=torch.Generator().manual_seed(8))).to(dtype)
    out, w = run_decode(pool, q, window, n_sink, record=True)
    assert Bd.device_error() == 0
    pool.table = full
    check_decode(pool, q, window, n_sink, out, w)


@pytest.mark.gpu
def test_decode_bad_tables_and_lengths_are_reported(cuda_device):
    pool = Pool(2, 128, 16, (200, 90), BF, seed=9)
    q = torch.randn(2, 8, 1, 128).to(BF)
    good, _ = run_decode(pool, q)
    assert Bd.device_error() == 0
    for value in (-1, pool.k.shape[0], 1 << 30):
        table = pool.table.clone()
        table[0, 3] = value
        keep, pool.table = pool.table, table
        out, w = run_decode(pool, q, record=True)
        pool.table = keep
        assert Bd.device_error() == 4
        assert torch.equal(out[1], good[1])
        j = torch.arange(200)
        seen = ((j < 48) | (j >= 64)).expand(4, 200)       # the bad page's keys are not seen
        for g in range(2):
            k, v = R.gather_pages(pool.k, keep[0], 200)[g], R.gather_pages(pool.v, keep[0], 200)[g]
            o, mag, _, S = R.attend(q[0, 4 * g:4 * g + 4, 0].double(), k.double(), v.double(), seen)
            R.assert_close(out[0, 4 * g:4 * g + 4, 0], o, R.out_tol(o, mag, S, 128, 184, BF), "bad page")
    pool.seq_len = torch.tensor([300, -5], dtype=torch.int32)
    out, _ = run_decode(pool, q, max_len=200)
    assert Bd.device_error() == 4
    assert torch.equal(out[0], good[0]) and not out[1].any()


@pytest.mark.gpu
def test_decode_large_batch(cuda_device):
    lens = [(37 * i) % 211 for i in range(300)]
    pool = Pool(2, 64, 16, lens, BF, seed=10)
    q = torch.randn(300, 8, 1, 64, generator=torch.Generator().manual_seed(11)).to(BF)
    out, w = run_decode(pool, q, record=True)
    assert Bd.device_error() == 0
    check_decode(pool, q, None, 0, out, w)


@pytest.mark.gpu
def test_decode_shared_pages(cuda_device):
    """Two sequences share their first pages (a common prompt): both read them, and the record
    gets both sums."""
    pool = Pool(2, 128, 16, (64, 40), F32, seed=12)
    pool.table[1, :2] = pool.table[0, :2]
    q = torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(13))
    out, w = run_decode(pool, q, record=True)
    ref, tol, rw, we = decode_ref(pool, q, 1 << 20, 0)
    R.assert_close(out, ref, tol, "out")
    got = R.gather_pages(w, pool.table[0], 32).double() - R.gather_pages(pool.w, pool.table[0], 32).double()
    R.assert_close(got, rw[0][:, :32] + rw[1][:, :32], we[0][:, :32] + we[1][:, :32] + 3 * 2.0 ** -23, "shared record")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_decode_is_repeatable_in_a_graph_over_growing_sequences(dtype, cuda_device):
    pool = Pool(2, 128, 16, (900, 333, 0), dtype, seed=14)
    q = torch.randn(3, 8, 1, 128, generator=torch.Generator().manual_seed(15)).to(dtype)
    k, v, table, lens = pool.gpu()
    qg, w = q.cuda(), pool.w.cuda()
    out = torch.empty_like(qg)
    Bd.paged_decode_attn(qg, k, v, table, lens, 900)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Bd.paged_decode_attn(qg, k, v, table, lens, 900, weight_pages=w, out=out)
    for now in ((900, 333, 0), (129, 333, 0), (1, 0, 0)):
        pool.lens = list(now)
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        w.copy_(pool.w)
        graph.replay()
        torch.cuda.synchronize()
        a, aw = out.cpu(), w.cpu()
        w.copy_(pool.w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), a) and torch.equal(w.cpu().nan_to_num(7), aw.nan_to_num(7))
        check_decode(pool, q, None, 0, a, aw)
    assert Bd.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_decode_visible_bad_values_are_passed_on(dtype, bad, cuda_device):
    pool = Pool(2, 128, 16, (300, 300), dtype, seed=16)
    q = torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(17)).to(dtype)
    good, _ = run_decode(pool, q)
    pool.v[pool.table[0, 5].long(), 1, 3, 9] = bad
    out, _ = run_decode(pool, q)
    assert torch.equal(out[1], good[1]) and torch.equal(out[0, :4], good[0, :4])
    assert not torch.isfinite(out[0, 4:, 0, 9].float()).any()
    assert torch.isfinite(out[0, 4:, 0, :9].float()).all() and torch.isfinite(out[0, 4:, 0, 10:].float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [100, 3000])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_decode_bad_query_is_its_own_affair(dtype, n, cuda_device):
    pool = Pool(2, 128, 16, (n, n), dtype, seed=40)
    q = torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(41)).to(dtype)
    good, _ = run_decode(pool, q)
    q2 = q.clone()
    q2[0, 6, 0, 100] = float("nan")
    out, _ = run_decode(pool, q2)
    assert out[0, 6].isnan().all()
    out[0, 6] = good[0, 6]
    assert torch.equal(out, good)


# ---- append -----------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,page,n,start,counts", [
    (64, 8, 1, (0, 7, 8, 100), None), (128, 16, 1, (0, 15, 16, 31), (1, 0, 1, 1)),
    (128, 24, 77, (5, 0, 200, 23), None), (64, 64, 300, (0, 1, 63, 64), (300, 1, 0, 299)),
    (128, 1024, 33, (1000, 0, 1023, 5), None)])
def test_append(d, page, n, start, counts, dtype, cuda_device):
    cnt = counts or (n,) * 4
    pool = Pool(3, d, page, [s + c for s, c in zip(start, cnt)], dtype, seed=18)
    g = torch.Generator().manual_seed(19)
    kn, vn = torch.randn(4, 3, n, d, generator=g).to(dtype), torch.randn(4, 3, n, d, generator=g).to(dtype)
    k, v, table, _ = pool.gpu()
    w = pool.w.cuda()
    Bd.paged_append(kn.cuda(), vn.cuda(), k, v, table, torch.tensor(start, dtype=torch.int32).cuda(),
                    n_new=None if counts is None else torch.tensor(cnt, dtype=torch.int32).cuda(), weight_pages=w)
    assert Bd.device_error() == 0
    for b in range(4):
        j = torch.arange(start[b], start[b] + cnt[b])
        at = (pool.table[b][j // page].long(), slice(None), j % page)
        pool.k[at] = kn[b, :, :cnt[b]].transpose(0, 1)
        pool.v[at] = vn[b, :, :cnt[b]].transpose(0, 1)
        pool.w[at] = 0
    same = lambda x, y: torch.equal(x.cpu().float().nan_to_num(77), y.float().nan_to_num(77))   # noqa: E731
    assert same(k, pool.k) and same(v, pool.v) and same(w, pool.w)


@pytest.mark.gpu
def test_append_out_of_range_is_reported_and_not_written(cuda_device):
    pool = Pool(2, 64, 8, (24, 24), F32, seed=20)
    k, v, table, _ = pool.gpu()
    table[1, 1] = pool.k.shape[0]
    was = k.clone()
    kn = torch.randn(2, 2, 8, 64).cuda()
    Bd.paged_append(kn, kn, k, v, table, torch.tensor([24, 8], dtype=torch.int32).cuda())
    assert Bd.device_error() == 4
    Bd.paged_append(kn, kn, k, v, table, torch.tensor([-8, 2147483640], dtype=torch.int32).cuda())
    assert Bd.device_error() == 4
    assert torch.equal(k.nan_to_num(7), was.nan_to_num(7))


# ---- eviction -----------------------------------------------------------------------------

def run_evict(pool, budget, n_sink, n_recent, b_max=None):
    h_kv, page = pool.k.shape[1], pool.page
    kept = [min(n, c) for n, c in zip(pool.lens, budget)]
    b_max = b_max or max(max(budget), 1)
    dst = torch.full((len(kept), -(-b_max // page)), -1, dtype=torch.int32)
    free = list(pool.free)
    for b, m in enumerate(kept):
        for i in range(-(-m // page)):
            dst[b, i] = free.pop()
    k, v, table, lens = pool.gpu()
    w = pool.w.cuda()
    idx, new = Bd.paged_evict(k, v, w, table, lens, max(max(pool.lens), 1), torch.tensor(budget, dtype=torch.int32).cuda(),
                              b_max, dst.cuda(), n_sink=n_sink, n_recent=n_recent)
    assert Bd.device_error() == 0
    assert new.cpu().tolist() == kept
    idx = idx.cpu()
    for b, n in enumerate(pool.lens):
        m = kept[b]
        assert (idx[b, :, m:] == -1).all()
        for g in range(h_kv):
            rec = R.gather_pages(pool.w, pool.table[b], n)[g] if n else torch.zeros(0)
            rows = R.evict_rows(rec, n, budget[b], n_sink, n_recent)
            assert idx[b, g, :m].tolist() == rows, (b, g)
        if m:
            i = torch.arange(m)
            at = (dst[b][i // page].long(), slice(None), i % page)
            for t in (pool.k, pool.v, pool.w):
                src = R.gather_pages(t, pool.table[b], n)
                t[at] = torch.stack([src[g, idx[b, g, :m].long()] for g in range(h_kv)], 1)
    for got, want in ((k, pool.k), (v, pool.v), (w, pool.w)):
        assert torch.equal(got.cpu().float().nan_to_num(77), want.float().nan_to_num(77))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("page,lens,budget,n_sink,n_recent", [
    (8, (300, 41, 40, 1, 0), (40,) * 5, 2, 9),
    (16, (1000, 999, 17), (128, 1, 17), 0, 0),
    (24, (700, 64), (500, 0), 4, 64),
    (64, (2000,), (100,), 100, 50),          # the first tokens fill the budget
    (64, (2000,), (100,), 30, 500),          # the rest of it goes to the latest
    (128, (5000, 4000), (4999, 1), 1, 0),
])
def test_evict(page, lens, budget, n_sink, n_recent, dtype, cuda_device):
    pool = Pool(2, 64 if page < 64 else 128, page, lens, dtype, seed=21, spare=1 + sum(-(-c // page) for c in budget))
    run_evict(pool, budget, n_sink, n_recent)


@pytest.mark.gpu
def test_evict_ties_and_odd_records(cuda_device):
    """Equal records go to the lower position; -0 equals +0; infinities order; NaN ranks with
    -infinity."""
    pool = Pool(2, 64, 16, (600, 600), F32, seed=22, spare=20)
    pool.w.copy_(torch.where(pool.w.isnan(), pool.w, (pool.w * 4).floor()))
    pool.w[pool.table[0, 2].long(), 0, :6] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -3.0])
    pool.w[pool.table[1].long()] = 0.0
    run_evict(pool, (130, 77), 3, 11, b_max=200)


@pytest.mark.gpu
@pytest.mark.parametrize("h_kv,B,n", [(1, 1, 60000), (8, 1, 9000), (8, 2, 9000), (8, 4, 3000), (8, 8, 3000),
                                      (2, 80, 500), (1, 1, 200000), (4, 32, 30000)])
def test_evict_launch_forms(h_kv, B, n, cuda_device):
    """Rows over clusters of 16 CTAs down to one."""
    page, budget = 64, n // 7
    pool = Pool(h_kv, 64, page, (n,) * B, BF, seed=23, spare=1 + B * -(-budget // page))
    run_evict(pool, (budget,) * B, 4, 33)


# ---- the three together -----------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_generation_over_a_cache_that_is_kept_small(dtype, cuda_device):
    """A prompt, decode steps that record weights, an eviction, and more steps: every step's
    output against the 64-bit form over the rows the cache should hold."""
    B, h_q, h_kv, d = 3, 8, 2, 128
    g = torch.Generator().manual_seed(24)
    cache = Bd.PagedCache(B, h_q, h_kv, d, dtype, 60, 16, 20, "cuda", record=True)
    ks = [torch.zeros(h_kv, 0, d, dtype=dtype) for _ in range(B)]
    vs = [torch.zeros(h_kv, 0, d, dtype=dtype) for _ in range(B)]

    def append(n, counts=None):
        kn, vn = torch.randn(B, h_kv, n, d, generator=g).to(dtype), torch.randn(B, h_kv, n, d, generator=g).to(dtype)
        cache.append(kn.cuda(), vn.cuda(), counts)
        for b in range(B):
            c = n if counts is None else counts[b]
            ks[b], vs[b] = torch.cat([ks[b], kn[b, :, :c]], 1), torch.cat([vs[b], vn[b, :, :c]], 1)

    def step():
        append(1)
        q = torch.randn(B, h_q, 1, d, generator=g).to(dtype)
        out = cache.attend(q.cuda()).cpu()
        for b in range(B):
            n = ks[b].shape[1]
            assert cache.lens[b] == n
            for h in range(h_q):
                o, mag, _, S = R.attend(q[b, h].double(), ks[b][h // 4].double(), vs[b][h // 4].double(),
                                        torch.ones(1, n, dtype=torch.bool))
                R.assert_close(out[b, h], o, R.out_tol(o, mag, S, d, n, dtype), f"sequence {b} head {h}")

    append(200, [200, 77, 1])
    for _ in range(5):
        step()
    rec = [R.gather_pages(cache.weight_pages.cpu(), cache.block_table[b].cpu(), cache.lens[b]) for b in range(B)]
    for b in range(B):                         # 5 steps of h_q heads, a softmax each
        assert abs(float(rec[b].sum()) - 5 * h_q) < 1e-3
    idx = cache.evict([64, 50, 64], n_sink=4, n_recent=16).cpu()
    for b, m in enumerate((64, 50, 6)):
        assert cache.lens[b] == m
        for head in range(h_kv):
            rows = R.evict_rows(rec[b][head], rec[b].shape[1], (64, 50, 64)[b], 4, 16)
            assert idx[b, head, :m].tolist() == rows
        at = idx[b, :, :m].long()
        ks[b] = torch.stack([ks[b][h, at[h]] for h in range(h_kv)])
        vs[b] = torch.stack([vs[b][h, at[h]] for h in range(h_kv)])
    assert len(cache.free) + sum(map(len, cache.pages)) == 60
    for _ in range(20):
        step()
    assert Bd.device_error() == 0


@pytest.mark.gpu
def test_prompt_from_the_contiguous_cache_into_pages(cuda_device):
    """quoka_prefill writes a contiguous cache; its rows go into pages and a window call over
    the contiguous cache equals the paged one."""
    h_q, h_kv, d, C, n_chunks = 8, 2, 128, 64, 3
    g = torch.Generator().manual_seed(25)
    q = torch.randn(n_chunks, 1, h_q, C, d, generator=g).to(BF).cuda()
    kn = torch.randn(n_chunks, 1, h_kv, C, d, generator=g).to(BF).cuda()
    vn = torch.randn(n_chunks, 1, h_kv, C, d, generator=g).to(BF).cuda()
    n = n_chunks * C
    k, v = torch.zeros(h_kv, n, d, dtype=BF, device="cuda"), torch.zeros(h_kv, n, d, dtype=BF, device="cuda")
    idx = torch.zeros(1, h_kv, 64, dtype=torch.int32, device="cuda")
    Bd.quoka_prefill(q, kn, vn, k, v, (0, n), 16, (0, 64, 64), idx)
    cache = Bd.PagedCache(1, h_q, h_kv, d, BF, 16, 16, 16, "cuda")
    cache.append(k[None].contiguous(), v[None].contiguous())
    qt = torch.randn(1, h_q, 1, d, generator=g).to(BF).cuda()
    for window, n_sink in ((1000, 0), (50, 4)):
        a = cache.attend(qt, window=window, n_sink=n_sink)
        b = Bd.window_chunk_attn(qt, k, v, (0, n), (n - 1,), window, n_sink)
        assert torch.equal(a, b)


# ---- calls that a serving loop makes in other ways ------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_decode_largest_batch(dtype, cuda_device):
    lens = [(53 * i) % 97 for i in range(1023)] + [700]
    pool = Pool(1, 64, 8, lens, dtype, seed=30)
    q = torch.randn(1024, 4, 1, 64, generator=torch.Generator().manual_seed(31)).to(dtype)
    out, w = run_decode(pool, q, record=True)
    assert Bd.device_error() == 0
    check_decode(pool, q, None, 0, out, w)


@pytest.mark.gpu
def test_two_calls_at_once_on_two_streams(cuda_device):
    pools = [Pool(2, 128, 16, (3000, 77), BF, seed=32), Pool(2, 128, 16, (1200, 2500), BF, seed=33)]
    qs = [torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(34 + i)).to(BF) for i in range(2)]
    want = [run_decode(p, q)[0] for p, q in zip(pools, qs)]
    args = [(q.cuda(), *p.gpu()) for p, q in zip(pools, qs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [Bd.paged_decode_attn(q, k, v, t, n, max(p.lens), stream=s)
                for (q, k, v, t, n), p, s in zip(args, pools, streams)]
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o.cpu(), w)


@pytest.mark.gpu
def test_a_step_with_eviction_in_a_graph(cuda_device):
    """append, attention with the record and eviction captured once and replayed as the
    lengths change."""
    page, B, h_kv, d = 16, 2, 2, 128
    lens = (400, 399)
    pool = Pool(h_kv, d, page, [n + 40 for n in lens], BF, seed=36, spare=40)
    k, v, table, _ = pool.gpu()
    w = pool.w.nan_to_num(0.5).cuda()
    start = torch.tensor(lens, dtype=torch.int32).cuda()
    budget = torch.tensor([64, 64], dtype=torch.int32).cuda()
    dst = torch.tensor(pool.free[:8], dtype=torch.int32).view(2, 4).cuda()
    g = torch.Generator().manual_seed(37)
    kn, vn, q = (torch.randn(B, h, 1, d, generator=g).to(BF).cuda() for h in (h_kv, h_kv, 8))
    idx = torch.zeros(B, h_kv, 64, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    n1 = torch.empty_like(start)

    def step():
        Bd.paged_append(kn, vn, k, v, table, start, weight_pages=w)
        torch.add(start, 1, out=n1)
        Bd.paged_decode_attn(q, k, v, table, n1, 440, weight_pages=w, out=out)
        Bd.paged_evict(k, v, w, table, n1, 440, budget, 64, dst, n_sink=2, n_recent=8, idx_out=idx, new_len=new)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for now in (lens, (30, 439), (0, 63)):
        start.copy_(torch.tensor(now, dtype=torch.int32))
        w.copy_(torch.rand(w.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert Bd.device_error() == 0
        assert new.cpu().tolist() == [min(n + 1, 64) for n in now]
        for b, n in enumerate(now):
            rec = R.gather_pages(w.cpu(), table[b].cpu(), n + 1)
            ks, vs = (R.gather_pages(t.cpu(), table[b].cpu(), n + 1) for t in (k, v))
            assert torch.equal(ks[:, n], kn[b, :, 0].cpu()) and torch.equal(vs[:, n], vn[b, :, 0].cpu())
            m = min(n + 1, 64)
            for h in range(h_kv):
                rows = R.evict_rows(rec[h], n + 1, 64, 2, 8)
                assert idx[b, h, :m].tolist() == rows
                assert torch.equal(R.gather_pages(k.cpu(), dst[b].cpu(), m)[h], ks[h][rows])
            for h in range(8):
                o, mag, _, S = R.attend(q[b, h].cpu().double(), ks[h // 4].double(), vs[h // 4].double(),
                                        torch.ones(1, n + 1, dtype=torch.bool))
                R.assert_close(out[b, h].cpu(), o, R.out_tol(o, mag, S, d, n + 1, BF), f"length {n} head {h}")


@pytest.mark.gpu
def test_pools_past_32_bit_offsets(cuda_device):
    """Pools of more than 2^31 elements each, the sequence in their last pages."""
    page, h_kv, d, N = 64, 4, 128, 66000
    k, v = (torch.empty(N, h_kv, page, d, dtype=BF, device="cuda") for _ in range(2))
    w = torch.zeros(N, h_kv, page, device="cuda")
    assert k.numel() > 2 ** 31
    n = 300
    table = torch.tensor([[N - 1, N - 3, N - 2, N - 5, N - 4]], dtype=torch.int32)
    g = torch.Generator().manual_seed(38)
    kn, vn = (torch.randn(1, h_kv, n, d, generator=g).to(BF) for _ in range(2))
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    Bd.paged_append(kn.cuda(), vn.cuda(), k, v, table.cuda(), zero, weight_pages=w)
    q = torch.randn(1, 16, 1, d, generator=g).to(BF)
    ln = torch.tensor([n], dtype=torch.int32).cuda()
    out = Bd.paged_decode_attn(q.cuda(), k, v, table.cuda(), ln, n, weight_pages=w).cpu()
    for h in range(16):
        o, mag, _, S = R.attend(q[0, h].double(), kn[0, h // 4].double(), vn[0, h // 4].double(),
                                torch.ones(1, n, dtype=torch.bool))
        R.assert_close(out[0, h], o, R.out_tol(o, mag, S, d, n, BF), f"head {h}")
    dst = torch.tensor([[N - 7, N - 6]], dtype=torch.int32)
    idx, _ = Bd.paged_evict(k, v, w, table.cuda(), ln, n, torch.tensor([100], dtype=torch.int32).cuda(), 100, dst.cuda())
    rec = w[table[0].long().cuda()].transpose(0, 1).reshape(h_kv, -1)[:, :n].cpu()
    moved = k[dst[0].long().cuda()].transpose(0, 1).reshape(h_kv, -1, d)[:, :100].cpu()
    for h in range(h_kv):
        rows = R.evict_rows(rec[h], n, 100, 0, 0)
        assert idx[0, h].tolist() == rows
        assert torch.equal(moved[h], kn[0, h][rows])
    assert Bd.device_error() == 0


@pytest.mark.gpu
def test_counts_and_budgets_out_of_range_are_reported(cuda_device):
    pool = Pool(2, 64, 8, (24, 24), F32, seed=39, spare=10)
    k, v, table, lens = pool.gpu()
    kn = torch.randn(2, 2, 4, 64).cuda()
    Bd.paged_append(kn, kn, k, v, table, torch.tensor([0, 0], dtype=torch.int32).cuda(),
                    n_new=torch.tensor([9, -2], dtype=torch.int32).cuda())
    assert Bd.device_error() == 4
    assert torch.equal(R.gather_pages(k.cpu(), table[0].cpu(), 4), kn[0].cpu())
    assert torch.equal(R.gather_pages(k.cpu(), table[1].cpu(), 24), R.gather_pages(pool.k, pool.table[1], 24))
    dst = torch.tensor(pool.free[:2], dtype=torch.int32).view(2, 1).cuda()
    _, new = Bd.paged_evict(k, v, pool.w.cuda(), table, lens, 24, torch.tensor([50, -1], dtype=torch.int32).cuda(), 8, dst)
    assert Bd.device_error() == 4
    assert new.cpu().tolist() == [8, 0]


# ---- refusals (host checks) --------------------------------------------------------------------

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake device pointers are only passed where there is no GPU")
FAKE = 0x10000
SHAPE = dict(batch=2, h_q=8, h_kv=2, head_dim=128, dtype=Bd.QUOKA_BF16, page_size=16, num_pages=100, max_pages=10)
BAD_SHAPES = [
    (dict(head_dim=96), Bd.QUOKA_ERR_UNSUPPORTED), (dict(batch=0), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(batch=1025), Bd.QUOKA_ERR_UNSUPPORTED), (dict(h_q=9), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(h_q=130), Bd.QUOKA_ERR_UNSUPPORTED), (dict(dtype=9), Bd.QUOKA_ERR_UNSUPPORTED),
    (dict(page_size=0), Bd.QUOKA_ERR_UNSUPPORTED), (dict(page_size=12), Bd.QUOKA_ERR_UNSUPPORTED),
    (dict(page_size=2048), Bd.QUOKA_ERR_UNSUPPORTED), (dict(num_pages=0), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(max_pages=0), Bd.QUOKA_ERR_INVALID_ARG), (dict(num_pages=1 << 26), Bd.QUOKA_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 27), Bd.QUOKA_ERR_UNSUPPORTED),
]


def P(i):
    return FAKE + 0x1000 * i


def _append(s, kn=P(0), vn=P(1), n=4, k=P(2), v=P(3), rec=P(4), table=P(5), start=P(6), count=None):
    return Bd.lib().paged_append(ctypes.byref(s), kn, vn, n, k, v, rec, table, start, count, None)


def _decode(s, q=P(0), k=P(1), v=P(2), table=P(3), lens=P(4), max_len=160, window=160, n_sink=0, rec=None, out=P(5),
            ws=P(6) & ~255, ws_bytes=1 << 30):
    return Bd.lib().paged_decode_attn(ctypes.byref(s), q, k, v, table, lens, max_len, window, n_sink, rec, out, ws,
                                      ws_bytes, None)


def _evict(s, k=P(0), v=P(1), rec=P(2), table=P(3), lens=P(4), max_len=160, budget=P(5), b_max=64, n_sink=0, n_recent=0,
           dst=P(6), dst_pages=4, idx=P(7), new=P(8)):
    return Bd.lib().paged_evict(ctypes.byref(s), k, v, rec, table, lens, max_len, budget, b_max, n_sink, n_recent, dst,
                                dst_pages, idx, new, None)


@no_gpu
@pytest.mark.parametrize("call", [_append, _decode, _evict])
@pytest.mark.parametrize("shape,status", BAD_SHAPES)
def test_rejects_shapes(call, shape, status):
    assert call(Bd.QuokaPagedShape(**{**SHAPE, **shape})) == status
    assert Bd.lib().quoka_last_error().decode()


@no_gpu
@pytest.mark.parametrize("call,args,status", [
    (_append, dict(kn=None), Bd.QUOKA_ERR_INVALID_ARG), (_append, dict(start=None), Bd.QUOKA_ERR_INVALID_ARG),
    (_append, dict(k=P(2) + 8), Bd.QUOKA_ERR_INVALID_ARG), (_append, dict(k=P(3)), Bd.QUOKA_ERR_INVALID_ARG),
    (_append, dict(kn=P(2)), Bd.QUOKA_ERR_INVALID_ARG), (_append, dict(n=0), Bd.QUOKA_ERR_INVALID_ARG),
    (_append, dict(n=8193), Bd.QUOKA_ERR_UNSUPPORTED), (_append, dict(table=P(5) + 2), Bd.QUOKA_ERR_INVALID_ARG),
    (_decode, dict(lens=None), Bd.QUOKA_ERR_INVALID_ARG), (_decode, dict(out=P(0)), Bd.QUOKA_ERR_INVALID_ARG),
    (_decode, dict(out=P(2)), Bd.QUOKA_ERR_INVALID_ARG), (_decode, dict(rec=P(7) + 4), Bd.QUOKA_ERR_INVALID_ARG),
    (_decode, dict(max_len=0), Bd.QUOKA_ERR_INVALID_ARG), (_decode, dict(max_len=161), Bd.QUOKA_ERR_INVALID_ARG),
    (_decode, dict(window=0), Bd.QUOKA_ERR_INVALID_ARG), (_decode, dict(n_sink=-1), Bd.QUOKA_ERR_INVALID_ARG),
    (_decode, dict(ws=None), Bd.QUOKA_ERR_WORKSPACE), (_decode, dict(ws_bytes=64), Bd.QUOKA_ERR_WORKSPACE),
    (_decode, dict(ws=P(6) + 16), Bd.QUOKA_ERR_INVALID_ARG),
    (_evict, dict(rec=None), Bd.QUOKA_ERR_INVALID_ARG), (_evict, dict(dst=P(3)), Bd.QUOKA_ERR_INVALID_ARG),
    (_evict, dict(k=P(1)), Bd.QUOKA_ERR_INVALID_ARG), (_evict, dict(b_max=0), Bd.QUOKA_ERR_INVALID_ARG),
    (_evict, dict(b_max=65), Bd.QUOKA_ERR_INVALID_ARG), (_evict, dict(new=P(4)), Bd.QUOKA_ERR_INVALID_ARG),
    (_evict, dict(n_recent=-1), Bd.QUOKA_ERR_INVALID_ARG), (_evict, dict(idx=P(7) + 8), Bd.QUOKA_ERR_INVALID_ARG),
    (_evict, dict(max_len=161), Bd.QUOKA_ERR_INVALID_ARG),
])
def test_rejects_arguments(call, args, status):
    assert call(Bd.QuokaPagedShape(**SHAPE), **args) == status
    assert Bd.lib().quoka_last_error().decode()


@no_gpu
def test_evict_refuses_lengths_past_its_limit():
    big = Bd.QuokaPagedShape(**{**SHAPE, "max_pages": 100000, "num_pages": 100000})
    assert _evict(big, max_len=786433) == Bd.QUOKA_ERR_UNSUPPORTED


def test_workspace_size():
    s = Bd.QuokaPagedShape(**SHAPE)
    n = Bd.paged_decode_workspace_size(s, 160, False)
    assert n > 0 and n % 256 == 0
    # the record needs the logits of every key tile: 128 keys x 4 heads of a group, fp32
    assert Bd.paged_decode_workspace_size(s, 160, True) - n >= 4 * 2 * 128 * 4 * 4
    assert Bd.paged_decode_workspace_size(s, 161, False) == 0
    assert Bd.paged_decode_workspace_size(s, 0, False) == 0


def test_binding_refuses_mixed_tensors():
    k = torch.zeros(6, 2, 16, 64)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 1, 64)
    for bad in (dict(q=q.bfloat16()), dict(q=torch.zeros(2, 4, 1, 64)), dict(table=table.long()),
                dict(table=table.expand(3, 4)), dict(lens=torch.zeros(2, dtype=torch.int32)), dict(v=k[:5]),
                dict(v=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(w=torch.zeros(6, 2, 16).double()),
                dict(w=torch.zeros(6, 16, 2))):
        a = dict(q=q, k=k, v=k.clone(), table=table, lens=lens, w=None)
        a.update(bad)
        with pytest.raises(Bd.QuokaError):
            Bd.paged_decode_attn(a["q"], a["k"], a["v"], a["table"], a["lens"], 64, weight_pages=a["w"])
    with pytest.raises(Bd.QuokaError):
        Bd.paged_append(torch.zeros(1, 2, 3, 64), torch.zeros(1, 2, 4, 64), k, k.clone(), table, lens)
    with pytest.raises(Bd.QuokaError):
        Bd.paged_evict(k, k.clone(), torch.zeros(6, 2, 16), table, lens, 64, lens.float(), 8, table.clone())


def test_paged_cache_checks_its_pages():
    c = Bd.PagedCache(2, 4, 2, 64, F32, 4, 16, 3, "cpu")
    for counts, why in (([49, 0], "max_pages"), ([48, 17], "free"), ([-1, 0], "counts"), ([1], "counts")):
        with pytest.raises(Bd.QuokaError, match=why):
            c.append(torch.zeros(2, 2, 64, 64), torch.zeros(2, 2, 64, 64), counts)
    with pytest.raises(Bd.QuokaError, match="record"):
        c.evict(4)
    assert len(c.free) == 4 and c.lens == [0, 0]
