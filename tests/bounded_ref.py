"""Plain 64-bit forms of the window, paged-cache and eviction operators, and the bounds their
kernels are held to (CPU, torch float64; no code shared with the library).

Bounds.  A rounding is off by at most u = eps / 2 relative (bf16 2^-8, fp32 2^-24).
  logits   d products summed in fp32 and one scaling: off by at most (d + 4) 2^-24 S, S the
           largest sum |q_i k_i| / sqrt(d) of the row
  weights  p = e^(s - m) / l: the logit's and the maximum's error each enter once, plus 2^-18
           for the exponential, the sum and the division in fp32 (n terms of one sign: the
           sum is off by at most n 2^-24 relative)
  output   sum p v: the weights' error, one rounding of p to bf16 on the tensor-core path
           (u_bf16), the sum's own n 2^-24, all relative to sum p |v|; and one rounding of
           the result to its type, relative to |o|
"""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attend(q, k, v, seen):
    """q [R, d], k / v [n, d] float64, seen bool [R, n].  A key that is not seen takes no part,
    whatever it holds.  Returns out, sum p |v|, p and S per row; rows that see nothing: 0."""
    d = q.shape[1]
    x = (q @ k.T) / math.sqrt(d)
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True) if x.shape[1] else torch.full((q.shape[0], 1), -math.inf).double()
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    p = torch.where(seen, p, 0.0)
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / l, 0.0)
    out, mag = p @ v, p @ v.abs()
    S = torch.where(seen, (q.abs() @ k.abs().T) / math.sqrt(d), 0.0)
    S = S.amax(-1, keepdim=True) if x.shape[1] else torch.zeros(q.shape[0], 1).double()
    return out, mag, p, S


def weight_err(d, n, S):
    return 2 * (d + 4) * 2.0 ** -24 * S + 2.0 ** -18 + n * 2.0 ** -24


def out_tol(out, mag, S, d, n, dtype):
    pv = U[torch.bfloat16] if dtype == torch.bfloat16 else 0.0
    return mag * (weight_err(d, n, S) + pv + n * 2.0 ** -24) + out.abs() * U[dtype] + 1e-30


def assert_close(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst {float(err[bad].max()):.3g} "
                           f"over {float(tol.expand_as(err)[bad].min()):.3g}, first at {bad.nonzero()[0].tolist()}")


def window_seen(P, C, n, window, n_sink):
    """Which of n keys each of the chunk's queries sees."""
    j, at = torch.arange(n), torch.arange(P, P + C)[:, None]
    return (j <= at) & ((j < n_sink) | (j > at - window))


def gather_pages(pool, table_row, n):
    """Rows 0 .. n-1 of a sequence: pool [N, h_kv, ps, ...] -> [h_kv, n, ...]."""
    ps = pool.shape[2]
    j = torch.arange(n)
    return pool[table_row[j // ps].long(), :, j % ps].transpose(0, 1)


def evict_rows(weights, n, budget, n_sink, n_recent):
    """Kept positions of one (sequence, KV head): weights [n]."""
    kept = min(n, budget)
    first = min(n_sink, kept)
    last = min(n_recent, kept - first)
    mid = [-math.inf if math.isnan(w) else w for w in weights[first:n - last].tolist()]
    best = sorted(range(len(mid)), key=lambda i: (-mid[i], i))[:kept - first - last]
    return list(range(first)) + sorted(first + i for i in best) + list(range(n - last, n))
