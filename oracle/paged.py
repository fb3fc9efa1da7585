"""Rotary append to a paged cache and attention over it, restated in numpy.

The append is stated in fp32, one rounding per product and sum, because that is the operator's
definition (its stored bits are compared exactly); attention in fp64.
"""
from __future__ import annotations

import numpy as np


def positions(cu_q, kv_lens):
    """(request, position) of every row of the token arrays."""
    req, pos = [], []
    for b in range(len(kv_lens)):
        n = int(cu_q[b + 1] - cu_q[b])
        req += [b] * n
        pos += range(int(kv_lens[b]) - n, int(kv_lens[b]))
    return np.array(req, dtype=np.int64), np.array(pos, dtype=np.int64)


def rotate(x, rows, interleaved):
    """x fp32 [T][H][D], rows fp32 [T][rot] (cos then sin): the rotated fp32 elements."""
    x = np.array(x, dtype=np.float32)
    rot = rows.shape[1]
    c, s = rows[:, None, :rot // 2], rows[:, None, rot // 2:]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = x[..., ia], x[..., ib]
    y = x.copy()
    y[..., ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    y[..., ib] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return y


def gather(cache, table, n, page_size):
    """The first n slots of one request: cache [pages][page_size][H][D] -> [n][H][D]."""
    j = np.arange(n)
    return cache[np.asarray(table)[j // page_size], j % page_size]


def visible(n, kv, causal, window):
    """bool [n][kv]: which keys each new token of one request sees."""
    pos = (kv - n + np.arange(n))[:, None]
    j = np.arange(kv)[None, :]
    see = np.ones((n, kv), dtype=bool)
    if causal:
        see &= j <= pos
    if window:
        see &= j > pos - window
    return see


def attention(q, k, v, see, scale):
    """One request in fp64: q [n][Hq][D], k and v [kv][Hk][D], see [n][kv].

    Returns (out [n][Hq][D], lse [n][Hq], spread [n][Hq][D] = sum_j p_j |v_j|)."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.zeros((n, Hq, D))
    spread = np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    used = see.any(0)
    for h in range(Hq):
        kk, vv = k[used, h // G].astype(np.float64), v[used, h // G].astype(np.float64)
        x = q[:, h].astype(np.float64) @ kk.T * scale
        x = np.where(see[:, used], x, -np.inf)
        for i in range(n):
            if not see[i].any():
                continue
            m = x[i].max()
            p = np.exp(x[i] - m)
            lse[i, h] = m + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ vv
            spread[i, h] = p @ np.abs(vv)
    return out, lse, spread
