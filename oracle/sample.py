"""Sampling under temperature, top-k, top-p and min-p from given uniform numbers, in fp64."""
from __future__ import annotations

import numpy as np

FLUSH = 2.0 ** -41   # weights at or below this have no mass


def clean(z):
    z = np.asarray(z, dtype=np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    return np.minimum(z, float(np.finfo(np.float32).max))


def distribution(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Kept weights by index (0 where dropped), relative to the largest; None without a finite
    logit."""
    z = clean(z)
    V = len(z)
    if not (z > -np.inf).any():
        return None
    greedy = not temperature >= 1e-6
    T = 1.0 if greedy else min(temperature, 1e6)
    w = np.exp((z - z.max()) / T)
    w[w <= FLUSH] = 0.0
    order = np.lexsort((np.arange(V), -z))
    k = 1 if greedy else (top_k if 0 < top_k <= V else V)
    stay = order[:k]
    if not top_p >= 1.0:
        m = w[stay]
        before = np.concatenate([[0.0], np.cumsum(m)[:-1]])
        keep = before < max(top_p, 0.0) * m.sum()
        keep[0] = True
        stay = stay[keep]
    out = np.zeros(V)
    out[stay] = w[stay]
    if min_p > 0:
        out[out < min(min_p, 1.0)] = 0.0
    return out


def draw(weights, u):
    """The first index whose inclusive weight exceeds u of the whole."""
    cum = np.cumsum(weights)
    i = int(np.searchsorted(cum, u * cum[-1], side="right"))
    return min(i, int(np.flatnonzero(weights)[-1]))
