"""Edges of the window and paged-cache calls: tensors that are not on a GPU, calls that are
refused half way, caches without a free page, rows whose softmax has no finite logit, and what
the attention weights may be off by."""
import os

import pytest
import torch

import bounded_ref as R
from query_oriented_sparse_b200 import binding as Bd

BF, F32 = torch.bfloat16, torch.float32


# ---- tensors on the host ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_host_tensors_are_refused(dtype):
    """Every argument is right but for the device: refused before a kernel is given the pointers."""
    q, k, v = torch.zeros(1, 4, 8, 64, dtype=dtype), torch.zeros(1, 100, 64, dtype=dtype), torch.zeros(1, 100, 64, dtype=dtype)
    kp, vp, w = torch.zeros(6, 2, 16, 64, dtype=dtype), torch.zeros(6, 2, 16, 64, dtype=dtype), torch.zeros(6, 2, 16)
    table, lens = torch.arange(4, dtype=torch.int32)[None], torch.ones(1, dtype=torch.int32)
    rows = torch.zeros(1, 2, 3, 64, dtype=dtype)
    cache = Bd.PagedCache(1, 4, 2, 64, dtype, 6, 16, 4, "cpu", record=True)
    for call in (lambda: Bd.window_chunk_attn(q, k, v, (0, 100), (92,), 10),
                 lambda: Bd.window_chunk_attn(q[:, :, :1].contiguous(), k, v, (0, 100), (92,), 10),
                 lambda: Bd.paged_append(rows, rows.clone(), kp, vp, table, lens, weight_pages=w),
                 lambda: Bd.paged_decode_attn(q[:, :, :1].contiguous(), kp, vp, table, lens, 64, weight_pages=w),
                 lambda: Bd.paged_evict(kp, vp, w, table, lens, 64, lens, 8, table.clone()),
                 lambda: cache.append(rows, rows.clone()),
                 lambda: cache.attend(q[:, :, :1].contiguous())):
        with pytest.raises(Bd.QuokaError, match="not on a CUDA device") as e:
            call()
        assert e.value.status == Bd.QUOKA_ERR_INVALID_ARG


# ---- values that are not finite, all over the masked blocks ---------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_bad_values_in_every_masked_block(d, cuda_device):
    """Every seventh key holds NaN in one column of its own, so that each masked block of each tile
    is cleaned, by lanes all over its warps and in both halves of the columns.  A row has NaN in
    just the columns of the bad keys that it sees, and ten calls agree to the bit."""
    prefix, window, n_sink, C, h_q, h_kv = (700, 0, 333), 150, 5, 500, 16, 4
    g = torch.Generator().manual_seed(50)
    off = [0]
    for p in prefix:
        off.append(off[-1] + p + C)
    q = torch.randn(3, h_q, C, d, generator=g).to(BF)
    k, v = torch.randn(h_kv, off[-1], d, generator=g).to(BF), torch.randn(h_kv, off[-1], d, generator=g).to(BF)
    bad = torch.arange(0, off[-1], 7)
    col = (37 * torch.arange(bad.numel())) % d
    v[:, bad, col] = float("nan")
    has = torch.zeros(off[-1], d, dtype=torch.bool)
    has[bad, col] = True
    args = q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink
    first = Bd.window_chunk_attn(*args).cpu()
    for b, P in enumerate(prefix):
        j, at = torch.arange(P + C), torch.arange(P, P + C)[:, None]
        seen = (j <= at) & ((j < n_sink) | (j > at - window))
        want = (seen.float() @ has[off[b]:off[b] + P + C].float()) > 0
        assert torch.equal(first[b].isnan(), want.expand(h_q, C, d))
        assert not first[b].isinf().any()
    for _ in range(10):
        assert torch.equal(Bd.window_chunk_attn(*args).cpu().nan_to_num(77), first.nan_to_num(77))
    assert Bd.device_error() == 0


# ---- refused calls leave a paged cache as it was ----------------------------------------------------

def _state(c):
    return list(c.free), [list(p) for p in c.pages], list(c.lens), c.block_table.tolist(), c.seq_len.tolist()


def _refused_calls(c, dev):
    """Calls that pass the cache's own checks and are refused by the operator under it."""
    rows = lambda n, dt=BF, d=64: torch.zeros(2, 2, n, d, dtype=dt, device=dev)    # noqa: E731
    return [lambda: c.append(rows(40, F32), rows(40, F32)),                # another type
            lambda: c.append(rows(40), rows(39)),                          # k and v differ
            lambda: c.append(rows(40, d=128), rows(40, d=128)),
            lambda: c.append(rows(40)[0], rows(40)[0]),                    # a dimension is missing
            lambda: c.append(rows(40).transpose(2, 3).contiguous().transpose(2, 3), rows(40)),
            lambda: c.append(rows(9000), rows(9000), [40, 40]),            # more rows than a call takes
            lambda: c.evict(20, n_sink=-1),
            lambda: c.evict([20, 3], n_recent=-1)]


@pytest.mark.parametrize("i", range(8))
def test_refused_calls_leave_the_cache_on_the_host(i):
    """No GPU: the operators refuse every call, after the cache has looked for its pages."""
    c = Bd.PagedCache(2, 4, 2, 64, BF, 20, 16, 10, "cpu", record=True)
    c.pages, c.free, c.lens = [[0, 1], [2]], list(range(19, 2, -1)), [30, 5]
    c.block_table, c.seq_len = c._table(c.pages), torch.tensor(c.lens, dtype=torch.int32)
    was = _state(c)
    for _ in range(3):
        with pytest.raises(Bd.QuokaError):
            _refused_calls(c, "cpu")[i]()
        assert _state(c) == was


@pytest.mark.gpu
def test_refused_calls_leave_the_cache(cuda_device):
    """The same on the GPU; afterwards every page can still be had, and one more is refused."""
    c = Bd.PagedCache(2, 4, 2, 64, BF, 20, 16, 10, "cuda", record=True)
    one = lambda n: torch.ones(2, 2, n, 64, dtype=BF, device="cuda")       # noqa: E731
    c.append(one(30), one(30), [30, 5])
    was = _state(c)
    for call in _refused_calls(c, "cuda"):
        with pytest.raises(Bd.QuokaError):
            call()
        assert _state(c) == was
    c.append(one(130), one(130), [130, 123])
    assert len(c.free) == 2 and c.lens == [160, 128]
    was = _state(c)
    with pytest.raises(Bd.QuokaError, match="max_pages"):
        c.append(one(1), one(1))
    assert _state(c) == was
    c.evict(16)
    assert len(c.free) == 18 and c.lens == [16, 16]
    assert sorted(c.free + sum(c.pages, [])) == list(range(20)) and Bd.device_error() == 0


# ---- rows whose visible logits are all -infinity ----------------------------------------------------

def _minus_inf(k, rows):
    """Makes the logits of these rows of k [..., rows, d] -infinity for queries with q[..., 0] < 0."""
    k[..., rows, :] = 0.0
    k[..., rows, 0] = float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (4, 1, 64), (20, 1, 64), (48, 1, 128)])
@pytest.mark.parametrize("C", [1, 3, 90])
def test_window_rows_without_a_finite_logit(C, h_q, h_kv, d, dtype, cuda_device):
    """Where a query sees such keys only, the softmax is 0 / 0: NaN, whatever the chunk's length.
    Beside one finite logit they weigh nothing."""
    g = torch.Generator().manual_seed(60)
    for P, window, n_sink in ((300, 5, 0), (3000, 2500, 0), (3000, 2500, 2), (40, 1000, 0)):
        n = P + C
        q = torch.randn(1, h_q, C, d, generator=g).to(dtype)
        q[..., 0] = -1.0
        k, v = torch.randn(h_kv, n, d, generator=g).to(dtype), torch.randn(h_kv, n, d, generator=g).to(dtype)
        _minus_inf(k, slice(n_sink, n))
        out = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), (0, n), (P,), window, n_sink).cpu()
        if n_sink == 0:
            assert out.isnan().all(), (P, window)
        else:                                       # what a cache of the first tokens alone gives
            for h in range(h_q):
                ks, vs = k[h * h_kv // h_q, :n_sink].double(), v[h * h_kv // h_q, :n_sink].double()
                o, mag, _, S = R.attend(q[0, h].double(), ks, vs, torch.ones(C, n_sink, dtype=torch.bool))
                R.assert_close(out[0, h], o, R.out_tol(o, mag, S, d, n_sink, dtype), f"head {h}")
    assert Bd.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (4, 1, 64), (20, 1, 64), (48, 1, 128)])
@pytest.mark.parametrize("n", [1, 100, 700, 6000])
def test_decode_rows_without_a_finite_logit(n, h_q, h_kv, d, dtype, cuda_device):
    """Two sequences of such keys but for one key of the second, with and without a record; an
    empty third one gives zeros.  CTAs that hold none but -infinity must not spoil the join."""
    page = 16
    per = -(-n // page)
    g = torch.Generator().manual_seed(61)
    q = torch.randn(3, h_q, 1, d, generator=g).to(dtype)
    q[..., 0] = -1.0
    k = torch.randn(2 * per, h_kv, page, d, generator=g).to(dtype)
    v = torch.randn(2 * per, h_kv, page, d, generator=g).to(dtype)
    at = (n // 3) // page, (n // 3) % page          # the second sequence's finite key
    keep = k[per + at[0], :, at[1]].clone()
    _minus_inf(k, slice(None))
    k[per + at[0], :, at[1]] = keep
    table = torch.arange(3 * per, dtype=torch.int32).view(3, per).clamp(max=2 * per - 1).cuda()
    lens = torch.tensor([n, n, 0], dtype=torch.int32).cuda()
    for record in (False, True):
        w = torch.full((2 * per, h_kv, page), 5.0).cuda() if record else None
        out = Bd.paged_decode_attn(q.cuda(), k.cuda(), v.cuda(), table, lens, n, weight_pages=w).cpu()
        assert out[0].isnan().all() and not out[2].any()
        want = v[per + at[0], :, at[1]].repeat_interleave(h_q // h_kv, 0)
        assert torch.equal(out[1, :, 0], want)      # one weight of 1
        if record:
            w = w.cpu().transpose(0, 1).reshape(h_kv, 2, per * page)
            assert w[:, 0, :n].isnan().all() and (w[:, :, n:] == 5.0).all()
            ref = torch.full((n,), 5.0)
            ref[n // 3] += h_q // h_kv
            assert torch.equal(w[:, 1, :n], ref.expand(h_kv, n))
    assert Bd.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_decode_with_bad_pages_alone_gives_zeros(dtype, cuda_device):
    """Keys whose pages are not in the pools are not seen: a sequence without any other key."""
    k, v = torch.randn(9, 2, 16, 64).to(dtype).cuda(), torch.randn(9, 2, 16, 64).to(dtype).cuda()
    table = torch.tensor([[-1, 9, 100]], dtype=torch.int32).cuda()
    w = torch.full((9, 2, 16), 5.0).cuda()
    out = Bd.paged_decode_attn(torch.randn(1, 8, 1, 64).to(dtype).cuda(), k, v, table,
                               torch.tensor([40], dtype=torch.int32).cuda(), 40, weight_pages=w)
    assert Bd.device_error() == 4
    assert not out.any() and (w == 5.0).all()


# ---- what a weight may be off by --------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("place", range(8))
def test_weights_are_fp32_wherever_their_key_lies(place, d, cuda_device):
    """bf16 chunks: the sum of the weights, read off the result.

    Key 0 has logit 0, value 1 and weight 1, rounded to bf16 without an error; the keys at
    `place` (mod 8) have a logit x in [-5, 0] of each row's own and value 0, every other key a
    logit far below.  So the result is 1 / (1 + M e^x) in bf16.  x is exact in fp32 up to the
    scaling.  Relative errors before the last rounding: the exponent |x log2 e| <= 7.3 is off by
    4 2^-24 of itself (scale, its division and square root, one rounding), 7.3 ln 2 2^-22 < 2^-19.6
    of the weight; the exponential 2^-22; the sum (16 terms to an accumulator, 8 blocks, joins: 30
    roundings) 30 2^-24 < 2^-19; 1 / l and its product 2^-23: in all less than 2^-18.  The result
    is a rounding to bf16 of something in between, and rounding is monotone."""
    h_q, h_kv, C, P = 32, 2, 256, 448
    g = torch.Generator().manual_seed(70 + place)
    q = torch.zeros(1, h_q, C, d)
    q[..., 0] = -4 * torch.rand(1, h_q, C, generator=g)
    q[..., 1] = 1.0
    q[..., 2] = -torch.rand(1, h_q, C, generator=g)
    q = q.to(BF)
    k, v = torch.zeros(h_kv, P + C, d), torch.zeros(h_kv, P + C, d)
    k[:, 1:, 1] = -4096.0
    rows = torch.arange(place, P, 8)
    rows = rows[rows > 0]
    unit = 8.0 if d == 64 else 11.0
    k[:, rows, 0], k[:, rows, 1], k[:, rows, 2] = unit, 0.0, unit / 256
    k[:, 0], v[:, 0] = 0.0, 1.0
    out = Bd.window_chunk_attn(q.cuda(), k.to(BF).cuda(), v.to(BF).cuda(), (0, P + C), (P,), P + C, 0).cpu()
    x = (q[..., 0].double() * unit + q[..., 2].double() * (unit / 256)) / d ** 0.5
    ref = 1 / (1 + rows.numel() * torch.exp(x))[..., None]
    lo, hi = (ref * (1 - 2.0 ** -18)).to(BF), (ref * (1 + 2.0 ** -18)).to(BF)
    off = ~((lo <= out) & (out <= hi))
    assert not off.any(), f"{int(off.any(-1).sum())} of {h_q * C} rows"
    assert Bd.device_error() == 0


# ---- eviction from a cache without free pages ---------------------------------------------------------

def test_eviction_limit_is_the_headers():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "quoka.h")
    assert f"#define QUOKA_MAX_EVICT_LEN {Bd.QUOKA_MAX_EVICT_LEN}\n" in open(path).read()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("spare", [0, 2])
@pytest.mark.parametrize("lens,budget,n_sink,n_recent", [
    ((64, 40, 16, 100), [20, 40, 0, 17], 2, 5),      # one keeps everything, one nothing
    ((64, 40, 16, 100), [63, 39, 15, 99], 0, 0),     # as many pages as before
    ((700, 1, 0, 33), [333, 5, 7, 32], 40, 300),
])
def test_a_full_cache_is_evicted(lens, budget, n_sink, n_recent, spare, dtype, cuda_device):
    """Fewer free pages than the kept rows need: the same rows are kept as with free pages, the
    pages are given back, and the cache can be used on."""
    B, h_q, h_kv, d, page = len(lens), 8, 2, 128, 16
    g = torch.Generator().manual_seed(80)
    used = sum(-(-n // page) for n in lens)
    kn, vn = (torch.randn(B, h_kv, max(lens), d, generator=g).to(dtype) for _ in range(2))

    def filled(num_pages):
        c = Bd.PagedCache(B, h_q, h_kv, d, dtype, num_pages, page, 50, "cuda", record=True)
        c.append(kn.cuda(), vn.cuda(), lens)
        c.weight_pages.copy_(0)
        for b, n in enumerate(lens):
            w = torch.rand(h_kv, n, generator=torch.Generator().manual_seed(81 + b))
            j = torch.arange(n)
            c.weight_pages[c.block_table[b].cpu()[j // page].long().cuda(), :, (j % page).cuda()] = w.T.cuda()
        return c

    def rows(c):
        return [[R.gather_pages(t.cpu(), c.block_table[b].cpu(), n) if n else None for b, n in enumerate(c.lens)]
                for t in (c.k_pages, c.v_pages, c.weight_pages)]

    full, roomy = filled(used + spare), filled(4 * used)
    assert len(full.free) == spare < sum(-(-min(n, b) // page) for n, b in zip(lens, budget))
    was = _state(full)
    for bad in (dict(n_sink=-1), dict(n_recent=-1)):
        with pytest.raises(Bd.QuokaError) as e:
            full.evict(budget, **bad)
        assert e.value.status == Bd.QUOKA_ERR_INVALID_ARG and _state(full) == was
    before = rows(full)
    idx = full.evict(budget, n_sink=n_sink, n_recent=n_recent)
    assert torch.equal(idx, roomy.evict(budget, n_sink=n_sink, n_recent=n_recent))
    keep = [min(n, b) for n, b in zip(lens, budget)]
    for b, k in enumerate(keep):
        for h in range(h_kv):
            want = R.evict_rows(before[2][b][h], lens[b], budget[b], n_sink, n_recent) if lens[b] else []
            assert idx[b, h].tolist() == want + [-1] * (idx.shape[2] - k)
            for t, old in zip(rows(full), before):
                if k:
                    assert torch.equal(t[b][h], old[b][h][want])
    assert full.lens == keep and full.seq_len.tolist() == keep
    assert [len(p) for p in full.pages] == [-(-k // page) for k in keep]
    assert sorted(full.free + sum(full.pages, [])) == list(range(used + spare))
    assert full.block_table.tolist() == full._table(full.pages).tolist()
    q, new = torch.randn(B, h_q, 1, d, generator=g).to(dtype).cuda(), kn[:, :, :1].contiguous().cuda()
    counts = [1 if k % page else 0 for k in keep]    # (the second case leaves no page free)
    for c in (full, roomy):
        c.append(new, new, counts)
    assert torch.equal(full.attend(q), roomy.attend(q))
    assert Bd.device_error() == 0


# ---- counts past 32 bits --------------------------------------------------------------------------------

def test_sizes_past_32_bits_on_the_host():
    shape = Bd.make_shape(1, 8, 2, 128, 16, BF)
    most = Bd.window_workspace_size(shape, 5000, 2 ** 31 - 1)
    assert most > 0 and Bd.window_workspace_size(shape, 5000, 2 ** 32 + 10) == most
    assert Bd.window_workspace_size(shape, 5000, -2 ** 32 + 10) == 0
    pages = Bd.QuokaPagedShape(2, 8, 2, 128, Bd.QUOKA_BF16, 16, 100, 10)
    assert Bd.paged_decode_workspace_size(pages, 2 ** 32 + 160, False) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("C", [1, 20])
def test_counts_past_32_bits(C, cuda_device):
    """A window or a number of first tokens of more than 2^31 keys is all of them, not its low
    32 bits; a length or budget of that size is refused."""
    g = torch.Generator().manual_seed(90)
    P, n = 300, 300 + C
    q = torch.randn(1, 8, C, 64, generator=g).to(BF).cuda()
    k, v = (torch.randn(2, n, 64, generator=g).to(BF).cuda() for _ in range(2))
    want = Bd.window_chunk_attn(q, k, v, (0, n), (P,), n)
    assert torch.equal(Bd.window_chunk_attn(q, k, v, (0, n), (P,), 2 ** 32 + 5), want)
    assert torch.equal(Bd.window_chunk_attn(q, k, v, (0, n), (P,), 3, n_sink=2 ** 32), want)
    c = Bd.PagedCache(1, 8, 2, 64, BF, 64, 16, 30, "cuda", record=True)
    c.append(k[None].contiguous(), v[None].contiguous())
    qt = q[:, :, -1:].contiguous()
    want = c.attend(qt)
    assert torch.equal(c.attend(qt, window=2 ** 32 + 5), want)
    assert torch.equal(c.attend(qt, window=3, n_sink=2 ** 32 + 1), want)
    args = c.k_pages, c.v_pages
    with pytest.raises(Bd.QuokaError):
        Bd.paged_decode_attn(qt, *args, c.block_table, c.seq_len, 2 ** 32 + n)
    with pytest.raises(Bd.QuokaError):
        Bd.paged_evict(*args, c.weight_pages, c.block_table, c.seq_len, n, c.seq_len, 8, c.block_table.clone(), n_sink=-2 ** 32)
    idx = c.evict(20, n_recent=2 ** 32 + 1)
    assert idx[0, 0].tolist() == list(range(n - 20, n)) and Bd.device_error() == 0


# ---- what the weight record must leave alone ------------------------------------------------------------

UNUSED = 77.0


def _recorded(dtype, h_q, h_kv, d, page, lens, table_of=None, window=None, n_sink=0):
    """Attention over pools whose record holds UNUSED in every slot without a key: the record
    before and after, [page, head, slot], on the CPU, and the 64-bit weights per sequence."""
    g = torch.Generator().manual_seed(100)
    per = [-(-n // page) for n in lens]
    N = sum(per) + 4
    perm = torch.randperm(N, generator=g).tolist()
    table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32)
    was = torch.full((N, h_kv, page), UNUSED)
    for b, (n, m) in enumerate(zip(lens, per)):
        pages = [perm.pop() for _ in range(m)]
        table[b, :m] = torch.tensor(pages, dtype=torch.int32)
        j = torch.arange(n)
        was[table[b][j // page].long(), :, j % page] = torch.rand(n, h_kv, generator=g)
    k, v = torch.randn(N, h_kv, page, d, generator=g).to(dtype), torch.randn(N, h_kv, page, d, generator=g).to(dtype)
    q = torch.randn(len(lens), h_q, 1, d, generator=g).to(dtype)
    given = table if table_of is None else table_of(table.clone())
    w = was.cuda()
    Bd.paged_decode_attn(q.cuda(), k.cuda(), v.cuda(), given.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                         max(max(lens), 1), window=window, n_sink=n_sink, weight_pages=w)
    want, tol = was.double(), torch.zeros(was.shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        there = (given[b][j // page] >= 0) & (given[b][j // page] < N)
        seen = there & ((j < n_sink) | (j >= n - (window or n)))
        if not seen.any():
            continue
        j = j[seen]
        for h in range(h_kv):
            kk = k[table[b][j // page].long(), h, j % page].double()
            G = h_q // h_kv
            _, _, p, S = R.attend(q[b, h * G:(h + 1) * G, 0].double(), kk, kk, torch.ones(G, j.numel(), dtype=torch.bool))
            at = table[b][j // page].long(), h, j % page
            want[at] += p.sum(0)
            # each head's weight, the sum over the heads, and the addition in memory
            tol[at] = (p * R.weight_err(d, j.numel(), S)).sum(0) + G * 2.0 ** -24 * p.sum(0) + want[at] * 2.0 ** -24
    return was, w.cpu(), want, tol


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (4, 1, 64), (5, 1, 128), (20, 1, 64), (64, 1, 128)])
@pytest.mark.parametrize("page,lens,window,n_sink", [
    (8, (1, 7, 0, 300), None, 0), (16, (2000, 5, 131), None, 0), (24, (700, 9), 100, 5),
    (256, (257, 255, 256), None, 0), (16, (9000,), 3000, 40), (16, tuple(range(1, 200, 3)), 50, 1)])
def test_record_changes_visible_keys_only(page, lens, window, n_sink, h_q, h_kv, d, dtype, cuda_device):
    was, w, want, tol = _recorded(dtype, h_q, h_kv, d, page, lens, window=window, n_sink=n_sink)
    assert Bd.device_error() == 0
    assert torch.equal(w[tol == 0], was[tol == 0])          # to the bit: unseen, unused and spare slots
    R.assert_close(w, want, tol, "record")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [-1, 1 << 30, "pages"])
@pytest.mark.parametrize("lens", [(200, 90), (6000, 90)])
def test_record_beside_a_bad_page(lens, value, dtype, cuda_device):
    """The keys of a page that is not in the pools take no weight and get none; everybody else's
    weights are what they are without those keys."""
    def table_of(t):
        t[0, 3] = sum(-(-n // 16) for n in lens) + 4 if value == "pages" else value
        return t

    was, w, want, tol = _recorded(dtype, 8, 2, 128, 16, lens, table_of)
    assert Bd.device_error() == 4
    assert torch.equal(w[tol == 0], was[tol == 0])
    R.assert_close(w, want, tol, "record")
    assert int((tol[:, 0] != 0).sum()) == sum(lens) - 16


# ---- chunks that see more first tokens than latest ones ---------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("h_q,h_kv,d,C,prefix,window,n_sink,split", [
    (32, 8, 128, 2, (3000,), 64, 2000, False),       # whole tiles: the window alone is short
    (8, 2, 64, 2, (3000, 1500), 64, 2000, False),
    (8, 2, 128, 9, (5000,), 1100, 3333, True),        # units of first tokens only, of both, of the window only
    (8, 2, 64, 9, (5000, 3500), 1100, 2000, True),
    (4, 4, 128, 40, (4000,), 1200, 2701, True),
])
def test_mostly_first_tokens(h_q, h_kv, d, C, prefix, window, n_sink, split, dtype, cuda_device):
    shape = Bd.make_shape(len(prefix), h_q, h_kv, d, C, dtype)
    assert (Bd.window_workspace_size(shape, max(prefix), window) > 0) == split
    g = torch.Generator().manual_seed(110)
    off = [0]
    for p in prefix:
        off.append(off[-1] + p + C)
    q = torch.randn(len(prefix), h_q, C, d, generator=g).to(dtype)
    k, v = (torch.randn(h_kv, off[-1], d, generator=g).to(dtype) for _ in range(2))
    out = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink).cpu()
    assert Bd.device_error() == 0
    for b, P in enumerate(prefix):
        seen = R.window_seen(P, C, P + C, window, n_sink)
        for h in range(h_q):
            ks, vs = (t[h * h_kv // h_q, off[b]:off[b + 1]].double() for t in (k, v))
            o, mag, _, S = R.attend(q[b, h].double(), ks, vs, seen)
            R.assert_close(out[b, h], o, R.out_tol(o, mag, S, d, seen.sum(-1, keepdim=True), dtype), f"{b} {h}")
