"""Operators of a bounded or paged KV cache: what each computes in plain torch operations,
the calls that run it in the library, and the cases it is timed at.

    window    attention of a chunk (or of one new token) over a sliding window of the cache
              and a few first tokens that stay visible
    append    new K/V rows of a batch into the pages of a paged cache
    decode    attention of one new token per sequence over a paged cache, optionally adding
              every key's attention weight to a per-key record
    evict     per KV head, the rows of a paged cache with the most accumulated attention
              weight (plus the first and the latest ones) copied into fewer pages
"""
import math
import random

import torch

own = False          # true: run() makes the library's calls; false: the plain form

# (query heads, KV heads) of the repository's workloads and tests, from one group of 4 heads
# to groups of 16 and 1
HEADS = [(4, 1), (8, 2), (32, 8), (64, 8), (64, 4), (8, 8)]


def listed():
    return [
        # the 128K-context chunk step, attended through a 4K window and 64 first tokens
        dict(name="window_chunk_128k", op="window", batch=1, h_q=32, h_kv=8, d=128, dtype="bf16", chunk=4096,
             lo=131072, hi=131072, len_seed=3, window=4096, sink=64),
        # the ragged batch (8 sequences of 4K to 64K, 16 heads to a KV head), odd window
        dict(name="window_chunk_ragged", op="window", batch=8, h_q=64, h_kv=4, d=128, dtype="bf16", chunk=1024,
             lo=4096, hi=65536, len_seed=4, window=2047, sink=4),
        # a small fp32 step, sequences shorter and longer than the window: latency
        dict(name="window_chunk_small_f32", op="window", batch=3, h_q=4, h_kv=1, d=64, dtype="f32", chunk=100,
             lo=0, hi=400, len_seed=1, window=37, sink=4),
        # the 32-sequence decode step through a window
        dict(name="window_token_32", op="window", batch=32, h_q=32, h_kv=8, d=128, dtype="bf16", chunk=1,
             lo=2048, hi=16384, len_seed=5, window=2000, sink=4),
        # the 32-sequence decode step's new rows, and a prefill chunk's, into pages
        dict(name="append_token_32", op="append", batch=32, h_q=32, h_kv=8, d=128, dtype="bf16", page=16, new=1,
             lo=2048, hi=16384, len_seed=5, ragged=False),
        dict(name="append_chunk", op="append", batch=1, h_q=32, h_kv=8, d=128, dtype="bf16", page=64, new=4096,
             lo=131072, hi=131072, len_seed=3, ragged=False),
        # the 32-sequence decode step over all of its pages
        dict(name="decode_32", op="decode", batch=32, h_q=32, h_kv=8, d=128, dtype="bf16", page=16,
             lo=2048, hi=16384, len_seed=5, window=0, sink=0, weights=False),
        # one long sequence, its keys' weights recorded for a later eviction
        dict(name="decode_128k_weights", op="decode", batch=1, h_q=32, h_kv=8, d=128, dtype="bf16", page=64,
             lo=131072, hi=131072, len_seed=3, window=0, sink=0, weights=True),
        # two short fp32 sequences: latency
        dict(name="decode_small_f32", op="decode", batch=2, h_q=4, h_kv=1, d=64, dtype="f32", page=8,
             lo=1, hi=300, len_seed=2, window=0, sink=0, weights=True),
        # every sequence of the decode batch down to about 12 % of its longest
        dict(name="evict_32", op="evict", batch=32, h_q=32, h_kv=8, d=128, dtype="bf16", page=16,
             lo=2048, hi=16384, len_seed=5, budget=1984, sink=4, recent=64),
        # one long sequence down to an eighth, after its prompt
        dict(name="evict_128k", op="evict", batch=1, h_q=32, h_kv=8, d=128, dtype="bf16", page=64,
             lo=131072, hi=131072, len_seed=3, budget=16384, sink=64, recent=1024),
        # short fp32 sequences, some below their budget: latency
        dict(name="evict_small_f32", op="evict", batch=3, h_q=4, h_kv=1, d=64, dtype="f32", page=8,
             lo=1, hi=300, len_seed=6, budget=40, sink=2, recent=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "append", "decode", "decode", "evict"])
    h_q, h_kv = rng.choice(HEADS)
    c = dict(op=op, h_q=h_q, h_kv=h_kv, d=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
             batch=_log(rng, 1, 32), len_seed=rng.randrange(1 << 20))
    # keys of the whole batch and all KV heads, bounded by the largest listed cases'
    room = (2000000 if op == "window" else 1500000) // (c["batch"] * h_kv) // (2 if c["dtype"] == "f32" else 1)
    hi = _log(rng, 2, max(3, min(131072, room)))
    c["lo"], c["hi"] = rng.choice([hi, max(1, hi // 8), 1]), hi
    if op == "window":
        c["chunk"] = rng.choice([1, _log(rng, 1, 16), _log(rng, 16, 2048)])
        c["window"], c["sink"] = _log(rng, 1, 8192), rng.choice([0, 1, 4, _log(rng, 1, 300)])
        # logits of the plain form, bounded by a quarter of the largest listed case's (fp32: less)
        most = 250000000 if c["dtype"] == "bf16" else 60000000
        while c["chunk"] > 1 and c["batch"] * h_q * c["chunk"] * (c["chunk"] + min(c["window"], c["hi"]) + c["sink"]) > most:
            c["chunk"] = c["chunk"] // 2
        return c
    c["page"] = rng.choice([8, 16, 16, 24, 32, 64, 128, 256])
    if op == "append":
        c["new"] = rng.choice([1, _log(rng, 1, max(2, min(4096, 200000 // (c["batch"] * h_kv))))])
        c["ragged"] = c["new"] > 1 and rng.random() < 0.5
    elif op == "decode":
        c["window"], c["sink"] = rng.choice([(0, 0), (0, 0), (_log(rng, 1, hi), rng.choice([0, 4, 70]))])
        c["weights"] = rng.random() < 0.5
    else:
        c["budget"] = _log(rng, 1, max(2, hi // 2))
        c["sink"], c["recent"] = rng.choice([0, 4, 64]), rng.choice([0, 1, 64, 500])
    return c


def lens(c):
    """Tokens of each sequence before the step (window, append) or in the cache."""
    r = random.Random(c["len_seed"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _counts(c):
    """Rows of each sequence that an append writes."""
    r = random.Random(c["len_seed"] + 1)
    return [r.randint(1, c["new"]) if c["ragged"] else c["new"] for _ in range(c["batch"])]


def work(c):
    esz = 2 if c["dtype"] == "bf16" else 4
    row, n, g = c["d"] * esz, lens(c), c["h_kv"]
    if c["op"] == "window":
        C, W, S = c["chunk"], c["window"], c["sink"]
        seen = [sum(min(p + t + 1, min(W, p + t + 1) + min(S, max(0, p + t + 1 - W))) for t in range(C)) for p in n]
        rows = [C + min(p, W - 1) + min(S, max(0, p + 1 - W)) for p in n]
        return {"bytes": 2 * g * row * sum(rows) + 2 * c["batch"] * c["h_q"] * C * row,
                "flops": 4 * c["d"] * c["h_q"] * sum(seen)}
    if c["op"] == "append":
        return {"bytes": 4 * g * row * sum(_counts(c)) + 4 * g * sum(_counts(c)), "flops": 0}
    if c["op"] == "decode":
        W = c["window"] or c["hi"] + 1
        seen = sum(min(p, min(W, p) + min(c["sink"], max(0, p - W))) for p in n)
        return {"bytes": 2 * g * row * seen + 2 * c["batch"] * c["h_q"] * row + (8 * g * seen if c["weights"] else 0),
                "flops": 4 * c["d"] * c["h_q"] * seen}
    kept = sum(min(p, c["budget"]) for p in n)
    return {"bytes": 4 * g * sum(n) + (4 * g * row + 12 * g) * kept, "flops": 0}


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, n, g, d, B = _dtype(c), lens(c), c["h_kv"], c["d"], c["batch"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    # queries and keys share four directions per KV head, as in the repository's rank4 recipe
    basis = torch.linalg.qr(randn(g, d, 4))[0]

    def keys(*shape):      # [..., g, rows, d] with g at dim -3
        x = randn(*shape, d)
        return x.add_(2 * randn(*shape, 4) @ basis.mT).to(dt)

    def queries(rows):     # [B, h_q, rows, d]
        G = c["h_q"] // g
        x = randn(B, g, G * rows, d) + 2 * randn(B, g, G * rows, 4) @ basis.mT
        return x.view(B, g * G, rows, d).to(dt).contiguous()

    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=c, lens=n)
    if c["op"] == "window":
        off = [0]
        for p in n:
            off.append(off[-1] + p + c["chunk"])
        s.update(kv_off=off, q=queries(c["chunk"]), k=keys(g, off[-1]), v=randn(g, off[-1], d).to(dt),
                 off_dev=torch.tensor(off[:-1], device="cuda"), len_dev=torch.tensor(n, device="cuda"))
        return s
    ps = c["page"]
    extra = c["new"] if c["op"] == "append" else 0
    per = [-(-(p + extra) // ps) for p in n]
    out_per = [-(-min(p, c["budget"]) // ps) for p in n] if c["op"] == "evict" else [0] * B
    pages = sum(per) + sum(out_per) + 1
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).cpu().tolist()

    def table(counts):     # each sequence's pages, in order, then -1
        t = torch.full((B, max(max(counts), 1)), -1, dtype=torch.int32)
        for b, m in enumerate(counts):
            t[b, :m] = torch.tensor([perm.pop() for _ in range(m)], dtype=torch.int32)
        return t.cuda()

    s.update(k=keys(pages, g, ps), v=randn(pages, g, ps, d).to(dt), table=table(per), seq_len=torch.tensor(n, **i32),
             max_len=max(n), weights=None)
    if c["op"] == "append":
        s.update(k_new=keys(B, g, c["new"]), v_new=randn(B, g, c["new"], d).to(dt),
                 count=torch.tensor(_counts(c), **i32) if c["ragged"] else None,
                 weights=torch.rand(pages, g, ps, generator=gen, device="cuda"))
    elif c["op"] == "decode":
        s.update(q=queries(1))
        if c["weights"]:
            s["weights"] = torch.rand(pages, g, ps, generator=gen, device="cuda")
    else:
        # weights collected over a generation: a heavy tail, and keys that were never attended
        w = torch.exp(1.5 * randn(pages, g, ps))
        s.update(weights=w * (torch.rand(pages, g, ps, generator=gen, device="cuda") > 0.05),
                 budget=torch.full((B,), c["budget"], **i32), dst=table(out_per))
    return s


def run(s):
    c = s["case"]
    if own:
        from query_oriented_sparse_b200 import binding as Bd
        if c["op"] == "window":
            return Bd.window_chunk_attn(s["q"], s["k"], s["v"], s["kv_off"], s["lens"], c["window"], c["sink"])
        if c["op"] == "append":
            Bd.paged_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["seq_len"], n_new=s["count"],
                            weight_pages=s["weights"])
            return s["k"], s["v"], s["weights"]
        if c["op"] == "decode":
            out = Bd.paged_decode_attn(s["q"], s["k"], s["v"], s["table"], s["seq_len"], s["max_len"],
                                       window=c["window"] or None, n_sink=c["sink"], weight_pages=s["weights"])
            return (out, s["weights"]) if c["weights"] else out
        idx, new_len = Bd.paged_evict(s["k"], s["v"], s["weights"], s["table"], s["seq_len"], s["max_len"],
                                      s["budget"], c["budget"], s["dst"], n_sink=c["sink"], n_recent=c["recent"])
        return idx, new_len, s["k"], s["v"], s["weights"]
    return dict(window=plain_window, append=plain_append, decode=plain_decode, evict=plain_evict)[c["op"]](s)


# ---- plain forms ---------------------------------------------------------------------

def _attend(q, k, v, seen):
    """q [B, g, G*t, d], k / v [B, g, n, d], seen [B, 1, G*t, n]; also the weights."""
    x = (q @ k.mT) / math.sqrt(q.shape[-1])
    x = x.masked_fill_(~seen, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    return p @ v, p


def plain_window(s):
    c, q, P = s["case"], s["q"], s["len_dev"]
    B, hq, C, d = q.shape
    g, W, S = c["h_kv"], c["window"], c["sink"]
    span = min(W, max(s["lens"]) + 1) + C - 1
    dev = q.device
    first = torch.arange(S, device=dev).expand(B, S)
    near = P[:, None] + C - span + torch.arange(span, device=dev)
    pos = torch.cat([first, near], 1)                                    # [B, n] key positions
    there = torch.cat([first < P[:, None] + C, near >= S], 1) & (pos >= 0)
    rows = s["off_dev"][:, None] + torch.minimum(pos.clamp(min=0), (P + C - 1)[:, None])
    k = s["k"][:, rows].transpose(0, 1).float()
    v = s["v"][:, rows].transpose(0, 1).float()
    at = P[:, None] + torch.arange(C, device=dev)                        # [B, C] query positions
    seen = (pos[:, None] <= at[:, :, None]) & ((pos[:, None] < S) | (pos[:, None] > at[:, :, None] - W)) & there[:, None]
    G = hq // g
    seen = seen[:, None].expand(B, G, C, -1).reshape(B, 1, G * C, -1)
    o, _ = _attend(q.float().view(B, g, G * C, d), k, v, seen)
    return o.view(B, hq, C, d).to(q.dtype)


def _slots(table, ps, at):
    """Page and slot of positions `at` [B, n] (positions without a page: page 0)."""
    page = table.long().gather(1, torch.clamp(at // ps, max=table.shape[1] - 1)).clamp(min=0)
    return page, at % ps


def plain_append(s):
    c = s["case"]
    B, g, n, d = s["k_new"].shape
    j = torch.arange(n, device="cuda").expand(B, n)
    if s["count"] is not None:                                           # repeat the last row in place of the absent ones
        j = torch.minimum(j, s["count"].long()[:, None] - 1)
    page, slot = _slots(s["table"], c["page"], s["seq_len"].long()[:, None] + j)
    for pool, new in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
        pool[page[:, None], torch.arange(g, device="cuda")[:, None], slot[:, None]] = new.gather(
            2, j[:, None, :, None].expand(B, g, n, d))
    s["weights"][page[:, None], torch.arange(g, device="cuda")[:, None], slot[:, None]] = 0.0
    return s["k"], s["v"], s["weights"]


def plain_decode(s):
    c, q, L = s["case"], s["q"], s["max_len"]
    B, hq, _, d = q.shape
    g, W = c["h_kv"], c["window"] or L
    pos = torch.arange(L, device="cuda").expand(B, L)
    n = s["seq_len"].long()[:, None]
    seen = (pos < n) & ((pos < c["sink"]) | (pos >= n - W))
    page, slot = _slots(s["table"], c["page"], pos)
    k = s["k"][page, :, slot].transpose(1, 2).float()
    v = s["v"][page, :, slot].transpose(1, 2).float()
    o, p = _attend(q.float().view(B, g, hq // g, d), k, v, seen[:, None, None].expand(B, 1, hq // g, L))
    o = o.view(B, hq, 1, d).to(q.dtype)
    if not c["weights"]:
        return o
    flat = (page[:, None] * g + torch.arange(g, device="cuda")[:, None]) * c["page"] + slot[:, None]
    s["weights"].view(-1).scatter_add_(0, flat.reshape(-1), p.sum(2).reshape(-1))
    return o, s["weights"]


def plain_evict(s):
    c, L, m = s["case"], s["max_len"], s["case"]["budget"]
    B, g, ps = c["batch"], c["h_kv"], c["page"]
    n = s["seq_len"].long()[:, None]
    kept = torch.minimum(n, s["budget"].long()[:, None])
    first = torch.clamp(kept, max=c["sink"])
    last = torch.minimum(kept - first, torch.full_like(kept, c["recent"]))
    pos = torch.arange(L, device="cuda").expand(B, L)
    page, slot = _slots(s["table"], ps, pos)
    w = s["weights"][page, :, slot].transpose(1, 2)
    w = w.masked_fill(((pos < first) | (pos >= n - last))[:, None], math.inf).masked_fill((pos >= n)[:, None], -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    keep = torch.arange(L, device="cuda") < kept[:, None]
    where = torch.where(keep, order, L)
    where = torch.sort(where, dim=-1).values
    where = torch.cat([where, torch.full((B, g, m), L, device="cuda")], -1)[..., :m]
    idx = torch.where(where < L, where, -1).to(torch.int32)
    i = torch.minimum(torch.arange(m, device="cuda").expand(B, m), kept - 1)   # absent ones repeat the last
    src = where.gather(2, i[:, None].expand(B, g, m))
    sp = s["table"].long()[:, None].expand(B, g, -1).gather(2, src // ps)
    dp, ds = _slots(s["dst"], ps, i)
    heads = torch.arange(g, device="cuda")[:, None]
    for pool in (s["k"], s["v"], s["weights"]):
        pool[dp[:, None], heads, ds[:, None]] = pool[sp, heads, src % ps]
    return idx, kept[:, 0].to(torch.int32), s["k"], s["v"], s["weights"]


# ---- the definitions in 64 bits, one sequence and KV head at a time --------------------------

def exact(c, seed):
    s = prepare(c, seed)
    return dict(window=exact_window, append=exact_append, decode=exact_decode, evict=exact_evict)[c["op"]](s)


def _softmax_rows(q, k, v, seen):
    x = torch.einsum("rd,nd->rn", q, k) * q.shape[-1] ** -0.5
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    p = torch.softmax(x, -1)
    return p, torch.einsum("rn,nd->rd", p, v)


def exact_window(s):
    c, q = s["case"], s["q"]
    W, S, C = c["window"], c["sink"], c["chunk"]
    G = c["h_q"] // c["h_kv"]
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b, P in enumerate(s["lens"]):
        at = torch.arange(P, P + C, device="cuda")[:, None]
        j = torch.arange(P + C, device="cuda")
        j = j[(j < S) | (j > P - W)]
        seen = (j <= at) & ((j < S) | (at - j < W))
        for h in range(c["h_q"]):
            k = s["k"][h // G][s["kv_off"][b] + j].double()
            v = s["v"][h // G][s["kv_off"][b] + j].double()
            out[b, h] = _softmax_rows(q[b, h].double(), k, v, seen)[1]
    return out


def _place(table, b, ps, j):
    return table[b].long()[j // ps], j % ps


def exact_append(s):
    c = s["case"]
    k, v, w = s["k"].double(), s["v"].double(), s["weights"].double()
    for b, (p, m) in enumerate(zip(s["lens"], _counts(c))):
        page, slot = _place(s["table"], b, c["page"], torch.arange(p, p + m, device="cuda"))
        for g in range(c["h_kv"]):
            k[page, g, slot] = s["k_new"][b, g, :m].double()
            v[page, g, slot] = s["v_new"][b, g, :m].double()
            w[page, g, slot] = 0
    return k, v, w


def exact_decode(s):
    c, q = s["case"], s["q"]
    G = c["h_q"] // c["h_kv"]
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    w = s["weights"].double() if c["weights"] else None
    for b, n in enumerate(s["lens"]):
        j = torch.arange(n, device="cuda")
        if c["window"]:
            j = j[(j < c["sink"]) | (n - 1 - j < c["window"])]
        page, slot = _place(s["table"], b, c["page"], j)
        for g in range(c["h_kv"]):
            qs = q[b, g * G:(g + 1) * G, 0].double()
            p, o = _softmax_rows(qs, s["k"][page, g, slot].double(), s["v"][page, g, slot].double(),
                                 torch.ones(G, j.numel(), dtype=torch.bool, device="cuda"))
            out[b, g * G:(g + 1) * G, 0] = o
            if c["weights"]:
                w[page, g, slot] += p.sum(0)
    return (out, w) if c["weights"] else out


def exact_evict(s):
    c, m = s["case"], s["case"]["budget"]
    k, v, w = s["k"].double(), s["v"].double(), s["weights"].double()
    for b, n in enumerate(s["lens"]):
        B = min(n, m)
        first = min(c["sink"], B)
        last = min(c["recent"], B - first)
        for g in range(c["h_kv"]):
            page, slot = _place(s["table"], b, c["page"], torch.arange(n, device="cuda"))
            mid = s["weights"][page, g, slot][first:n - last].cpu().tolist()
            best = sorted(range(len(mid)), key=lambda i: (-mid[i], i))[:B - first - last]
            rows = list(range(first)) + sorted(first + i for i in best) + list(range(n - last, n))
            rows = torch.tensor(rows, device="cuda", dtype=torch.long)
            dp, ds = _place(s["dst"], b, c["page"], torch.arange(B, device="cuda"))
            sp, ss = _place(s["table"], b, c["page"], rows)
            k[dp, g, ds] = s["k"][sp, g, ss].double()
            v[dp, g, ds] = s["v"][sp, g, ss].double()
            w[dp, g, ds] = s["weights"][sp, g, ss].double()
    return None, None, k, v, w
