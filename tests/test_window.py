"""window_chunk_attn against the plain 64-bit form: windows from one key to all of them, first
tokens that join the window or not, sequences without a prefix, chunks of one and of odd
lengths, every group size class, and values that are not numbers where nothing may see them."""
import ctypes

import pytest
import torch

import bounded_ref as R
from query_oriented_sparse_b200 import binding as Bd

BF, F32 = torch.bfloat16, torch.float32


def make(h_q, h_kv, d, C, prefix, dtype, seed=0, slack=0):
    """q, k, v on the CPU and kv_off; `slack` rows behind each sequence hold NaN."""
    g = torch.Generator().manual_seed(seed)
    off = [0]
    for p in prefix:
        off.append(off[-1] + p + C + slack)
    q = (1.5 * torch.randn(len(prefix), h_q, C, d, generator=g)).to(dtype)
    k = torch.randn(h_kv, off[-1], d, generator=g).to(dtype)
    v = torch.randn(h_kv, off[-1], d, generator=g).to(dtype)
    for b, p in enumerate(prefix):
        for t in (k, v):
            t[:, off[b] + p + C:off[b + 1]] = float("nan")
    return q, k, v, off


def check(q, k, v, off, prefix, window, n_sink, got, rows=None):
    B, h_q, C, d = q.shape
    G = h_q // k.shape[0]
    for b, P in enumerate(prefix):
        n = P + C
        seen = R.window_seen(P, C, n, window, n_sink)
        any_seen = seen.any(0)
        for h in range(h_q):
            ks = k[h // G, off[b]:off[b] + n].double()[any_seen]
            vs = v[h // G, off[b]:off[b] + n].double()[any_seen]
            out, mag, _, S = R.attend(q[b, h].double(), ks, vs, seen[:, any_seen])
            tol = R.out_tol(out, mag, S, d, seen.sum(-1, keepdim=True), q.dtype)
            r = slice(None) if rows is None else rows
            R.assert_close(got[b, h][r], out[r], tol[r], f"sequence {b} head {h}")


CASES = [
    # h_q, h_kv, d, C, prefixes, window, n_sink
    (4, 1, 64, 100, (0, 37, 300), 37, 4),
    (4, 1, 128, 100, (0, 37, 300), 37, 4),
    (8, 2, 128, 65, (513,), 1, 0),                # only the own key
    (8, 2, 64, 65, (513,), 1, 3),
    (8, 2, 128, 257, (700, 129), 128, 130),       # first tokens over more than one block
    (8, 2, 64, 257, (700, 129), 128, 130),
    (2, 2, 128, 300, (64,), 100000, 0),           # every earlier key, one head per KV head
    (2, 2, 64, 300, (64,), 2147483647, 2147483647),
    (5, 1, 128, 70, (400,), 90, 7),               # a group that does not divide the tile
    (12, 2, 64, 70, (400,), 90, 7),
    (16, 1, 128, 33, (1000, 0, 5), 256, 16),
    (64, 1, 128, 9, (260,), 100, 1),
    (64, 1, 64, 9, (260,), 100, 1),
    (8, 2, 128, 2, (3000,), 2000, 4),             # a short chunk
    (4, 4, 128, 640, (640,), 640, 0),
    (8, 2, 128, 16, (5000, 0, 600), 4000, 70),    # tiles split over their keys, some with fewer keys than units
    (8, 2, 64, 16, (5000, 0, 600), 4000, 70),
    (32, 8, 128, 2, (3000, 2999), 2500, 4),
    (64, 1, 64, 3, (4000,), 100000, 0),
    (1, 1, 128, 1000, (500,), 300, 4),            # more units than streams
    (8, 8, 64, 3000, (0,), 200, 4),
]
TOKEN_CASES = [
    (4, 1, 64, (0, 1, 40, 300), 37, 4),
    (32, 8, 128, (2100, 0, 127, 128), 1000, 4),
    (8, 2, 128, (3000, 129), 1, 0),
    (5, 1, 128, (515, 64), 300, 260),
    (64, 1, 128, (4100,), 100000, 0),
    (64, 1, 64, (4100,), 700, 128),
    (20, 1, 64, (999, 3), 200, 5),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_chunk(case, dtype, cuda_device):
    h_q, h_kv, d, C, prefix, window, n_sink = case
    q, k, v, off = make(h_q, h_kv, d, C, prefix, dtype, slack=5)
    out = torch.full_like(q, float("nan")).cuda()
    Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink, out=out)
    assert Bd.device_error() == 0
    check(q, k, v, off, prefix, window, n_sink, out.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", TOKEN_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_token(case, dtype, cuda_device):
    h_q, h_kv, d, prefix, window, n_sink = case
    q, k, v, off = make(h_q, h_kv, d, 1, prefix, dtype, seed=1, slack=3)
    out = torch.full_like(q, float("nan")).cuda()
    Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink, out=out)
    assert Bd.device_error() == 0
    check(q, k, v, off, prefix, window, n_sink, out.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("C", [1, 150])
def test_expired_rows_are_not_used(C, d, dtype, cuda_device):
    """Rows between the first tokens and the oldest window hold NaN; nobody sees them."""
    prefix, window, n_sink = (900, 401), 200, 3
    q, k, v, off = make(8, 2, d, C, prefix, dtype, seed=2)
    for b, P in enumerate(prefix):
        for t in (k, v):
            t[:, off[b] + n_sink:off[b] + P - window + 1] = float("nan")
    out = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink)
    check(q, k, v, off, prefix, window, n_sink, out.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_rows_reach_only_their_readers(d, dtype, bad, cuda_device):
    """Some queries see the bad row, others do not: those get what they get without it, to the
    bit; and every query that sees a bad value of one dimension has it there and only there."""
    prefix, window, n_sink, C = (300, 0), 90, 0, 130
    q, k, v, off = make(8, 2, d, C, prefix, dtype, seed=3)
    clean = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink).cpu()
    for b, P in enumerate(prefix):
        for u in (40, 125):                              # chunk positions: the padded tail of a batch
            k2, v2 = k.clone(), v.clone()
            v2[:, off[b] + P + u, d - 3] = bad
            out = Bd.window_chunk_attn(q.cuda(), k2.cuda(), v2.cuda(), off, prefix, window, n_sink).cpu()
            t = torch.arange(C)
            sees = (t >= u) & (t - u < window)
            rest = torch.arange(d) != d - 3
            assert torch.equal(out[b][:, ~sees], clean[b][:, ~sees])
            assert torch.equal(out[1 - b], clean[1 - b])
            assert not torch.isfinite(out[b][:, sees, d - 3].float()).any()
            assert torch.isfinite(out[b][:, sees][..., rest].float()).all()
            if bad == bad:
                assert (out[b][:, sees, d - 3].float() == bad).all()
            k2[:, off[b] + P + u] = bad
            out = Bd.window_chunk_attn(q.cuda(), k2.cuda(), v2.cuda(), off, prefix, window, n_sink).cpu()
            assert torch.equal(out[b][:, ~sees], clean[b][:, ~sees])
    # an old row that the chunk's first queries still see
    P, b, u = 300, 0, 300 - 60
    v2 = v.clone()
    v2[:, off[b] + u, 5] = bad
    out = Bd.window_chunk_attn(q.cuda(), k.cuda(), v2.cuda(), off, prefix, window, n_sink).cpu()
    sees = P + torch.arange(C) - u < window
    assert torch.equal(out[b][:, ~sees], clean[b][:, ~sees])
    assert not torch.isfinite(out[b][:, sees, 5].float()).any()


@pytest.mark.gpu
@pytest.mark.parametrize("C", [1, 70])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_bad_query_is_its_own_affair(d, dtype, C, cuda_device):
    """A query that holds NaN gives NaN, and no other row changes."""
    prefix = (300, 41)
    q, k, v, off = make(8, 2, d, C, prefix, dtype, seed=9)
    clean = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, 200, 3).cpu()
    q2 = q.clone()
    q2[1, 5, C // 2, 3] = float("nan")
    out = Bd.window_chunk_attn(q2.cuda(), k.cuda(), v.cuda(), off, prefix, 200, 3).cpu()
    assert out[1, 5, C // 2].isnan().all()
    out[1, 5, C // 2] = clean[1, 5, C // 2]
    assert torch.equal(out, clean)


@pytest.mark.gpu
def test_all_keys_equal_selecting_every_key(cuda_device):
    """A window over everything is the attention of sparse_chunk_attn with every prefix key."""
    prefix, C = (500, 77), 140
    q, k, v, off = make(8, 2, 128, C, prefix, BF, seed=4)
    qc, kc, vc = q.cuda(), k.cuda(), v.cuda()
    idx = torch.full((2, 2, 500), -1, dtype=torch.int32)
    for b, P in enumerate(prefix):
        idx[b, :, :P] = torch.arange(P)
    a = Bd.sparse_chunk_attn(qc, kc, vc, off, prefix, prefix, idx.cuda())
    o = Bd.window_chunk_attn(qc, kc, vc, off, prefix, 1000)
    assert (a.float() - o.float()).abs().max() <= 2 ** -7 * a.float().abs().max()


@pytest.mark.gpu
def test_graph_replay_and_other_stream(cuda_device):
    prefix, window, n_sink = (700, 300), 250, 4
    for C in (1, 96):
        q, k, v, off = make(8, 2, 128, C, prefix, BF, seed=5)
        q, k, v = q.cuda(), k.cuda(), v.cuda()
        want = Bd.window_chunk_attn(q, k, v, off, prefix, window, n_sink)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = Bd.window_chunk_attn(q, k, v, off, prefix, window, n_sink, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        out = torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Bd.window_chunk_attn(q, k, v, off, prefix, window, n_sink, out=out)
        q2 = torch.randn_like(q.float()).to(BF)
        q.copy_(q2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, Bd.window_chunk_attn(q, k, v, off, prefix, window, n_sink))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_rows_in_split_tiles(d, dtype, cuda_device):
    """As above with each tile's keys split over several units."""
    prefix, window, n_sink, C = (2500,), 2000, 0, 12
    q, k, v, off = make(8, 2, d, C, prefix, dtype, seed=6)
    assert Bd.window_workspace_size(Bd.make_shape(1, 8, 2, d, C, dtype), 2500, window) > 0
    clean = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink).cpu()
    for at in (2500 + 7, 2500 - 1995, 2500 + 11):
        v2 = v.clone()
        v2[:, at, 11] = float("nan")
        out = Bd.window_chunk_attn(q.cuda(), k.cuda(), v2.cuda(), off, prefix, window, n_sink).cpu()
        p = 2500 + torch.arange(C)
        sees = (at <= p) & (at > p - window)
        assert 0 < int(sees.sum()) < C or at == 2500 + 11
        assert torch.equal(out[0][:, ~sees], clean[0][:, ~sees])
        assert out[0][:, sees, 11].isnan().all() and torch.isfinite(out[0][:, sees, :11].float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("C", [1, 40])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_long_prefix(dtype, C, cuda_device):
    prefix, window, n_sink = (120001,), 3001, 70
    q, k, v, off = make(4, 1, 64, C, prefix, dtype, seed=7)
    out = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink)
    check(q, k, v, off, prefix, window, n_sink, out.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("C", [1, 33])
def test_cache_past_32_bit_offsets(C, cuda_device):
    """A cache of more than 2^31 elements, the sequence in its last rows."""
    rows, P, d = 16800000, 500, 128
    q, k, v, _ = make(8, 1, d, C, (P,), BF, seed=8)
    kb, vb = (torch.empty(1, rows, d, dtype=BF, device="cuda") for _ in range(2))
    assert kb.numel() > 2 ** 31
    off = [0, rows - P - C, rows]
    kb[:, off[1]:], vb[:, off[1]:] = k.cuda(), v.cuda()
    whole = Bd.window_chunk_attn(q.cuda(), kb, vb, (off[1], rows), (P,), 200, 3)
    check(q, k, v, [0, P + C], (P,), 200, 3, whole.cpu())


# ---- refusals (host checks: no GPU needed, nothing is launched) --------------------------------

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake device pointers are only passed where there is no GPU")
FAKE = 0x10000


def _window(shape, q=FAKE, k=FAKE + 0x1000, v=FAKE + 0x2000, kv_off=(0, 1024), prefix=(512,), window=64, n_sink=4,
            out=FAKE + 0x3000, ws=FAKE, ws_bytes=1 << 30):
    return Bd.lib().window_chunk_attn(ctypes.byref(shape), q, k, v, Bd._host_i64(kv_off), Bd._host_i32(prefix),
                                      window, n_sink, out, ws, ws_bytes, None)


@no_gpu
@pytest.mark.parametrize("case,status", [
    (dict(shape=dict(head_dim=96)), Bd.QUOKA_ERR_UNSUPPORTED),
    (dict(shape=dict(batch=65)), Bd.QUOKA_ERR_UNSUPPORTED),
    (dict(shape=dict(h_q=7)), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(shape=dict(dtype=5)), Bd.QUOKA_ERR_UNSUPPORTED),
    (dict(window=0), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(window=-5), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(n_sink=-1), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(q=None), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(v=FAKE + 0x2004), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(out=FAKE), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(prefix=(900,)), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(prefix=(-1,)), Bd.QUOKA_ERR_INVALID_ARG),
    (dict(kv_off=(0, 1 << 31)), Bd.QUOKA_ERR_UNSUPPORTED),
    (dict(shape=dict(chunk=1), ws=None), Bd.QUOKA_ERR_WORKSPACE),
    (dict(shape=dict(chunk=1), ws_bytes=100), Bd.QUOKA_ERR_WORKSPACE),
    (dict(shape=dict(chunk=1), ws=FAKE + 64), Bd.QUOKA_ERR_INVALID_ARG),
])
def test_rejects(case, status):
    shp = dict(batch=1, h_q=8, h_kv=2, head_dim=128, chunk=256, dtype=Bd.QUOKA_BF16)
    shp.update(case.get("shape", {}))
    assert _window(Bd.QuokaShape(**shp), **{k: v for k, v in case.items() if k != "shape"}) == status
    assert Bd.lib().quoka_last_error().decode()


def test_workspace_size():
    for C, dtype, window in ((1, BF, 100), (1, F32, 100), (16, BF, 4096), (16, F32, 4096)):
        n = Bd.window_workspace_size(Bd.make_shape(2, 8, 2, 128, C, dtype), 4096, window)
        assert n > 0 and n % 256 == 0
    # one unit per tile: short windows, many tiles
    assert Bd.window_workspace_size(Bd.make_shape(2, 8, 2, 128, 64, BF), 4096, 100) == 0
    assert Bd.window_workspace_size(Bd.make_shape(8, 32, 8, 128, 4096, BF), 4096, 4096) == 0
    assert Bd.window_workspace_size(Bd.make_shape(2, 8, 2, 128, 4096, F32), 4096, 100) == 0
    assert Bd.window_workspace_size(Bd.make_shape(2, 8, 2, 96, 16, BF), 4096, 4096) == 0


def test_binding_refuses_strides_shapes_and_types():
    q, k, v = torch.zeros(1, 4, 8, 64), torch.zeros(1, 100, 64), torch.zeros(1, 100, 64)
    for bad in (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(v=v.bfloat16()), dict(k=k[:, :90]),
                dict(v=torch.zeros(1, 100, 128)[..., ::2]), dict(off=(0, 99)), dict(off=(0, 50, 100)),
                dict(q=q[0])):
        a = dict(q=q, k=k, v=v, off=(0, 100))
        a.update(bad)
        with pytest.raises(Bd.QuokaError):
            Bd.window_chunk_attn(a["q"], a["k"], a["v"], a["off"], (92,), 10)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_bad_key_reaches_every_reader(d, dtype, cuda_device):
    """A K row that holds NaN makes the rows that see it NaN, whichever of a block's keys it is."""
    prefix, window, C = (300,), 90, 130
    q, k, v, off = make(8, 2, d, C, prefix, dtype, seed=11)
    clean = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, 0).cpu()
    for u in range(16):
        k2 = k.clone()
        k2[:, 300 + 20 + u, 7] = float("nan")
        out = Bd.window_chunk_attn(q.cuda(), k2.cuda(), v.cuda(), off, prefix, window, 0).cpu()
        t = torch.arange(C)
        sees = (t >= 20 + u) & (t - 20 - u < window)
        assert out[0][:, sees].isnan().all()
        assert torch.equal(out[0][:, ~sees], clean[0][:, ~sees])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1e-3, 8.0, 40.0])
def test_flat_and_peaked_rows(scale, d, dtype, cuda_device):
    """From weights that are all alike to ones that leave the range of fp32."""
    prefix, window, n_sink, C = (500, 0), 333, 4, 200
    q, k, v, off = make(8, 2, d, C, prefix, dtype, seed=12)
    q = (scale * q.double()).to(dtype)
    out = Bd.window_chunk_attn(q.cuda(), k.cuda(), v.cuda(), off, prefix, window, n_sink).cpu()
    check(q, k, v, off, prefix, window, n_sink, out)
