"""Verification of drafted tokens against the target's probabilities, in fp64."""
from __future__ import annotations

import numpy as np

from . import sample


def shares(z, settings):
    """The row's probabilities under (temperature, top_k, top_p, min_p); zeros without a finite logit."""
    w = sample.distribution(z, *settings)
    return np.zeros(len(z)) if w is None else w / w.sum()


def proposal(V, token, y=None, settings=(1.0, 0, 1.0, 0.0), index=None):
    """What a draft was drawn from, over the target's V tokens: the drafter's row, or one token for certain."""
    q = np.zeros(V)
    if y is None:
        if 0 <= token < V:
            q[token] = 1.0
        return q, 1.0
    s = shares(y, settings)
    if index is None:
        q[:len(s)] = s
    else:
        index = np.asarray(index)
        has = (index >= 0) & (index < len(s))
        q[has] = s[index[has]]
    return q, (q[token] if 0 <= token < V else 0.0)


def ratio(p, given, token):
    """(p of the draft, the probability of accepting it)."""
    share = p[token] if 0 <= token < len(p) else 0.0
    if given > 0:
        return share, min(1.0, share / given)
    return share, 1.0 if share > 0 else 0.0


def rest(p, q):
    """What the next token is drawn from after a rejection, not normalised."""
    r = np.maximum(p - q, 0.0)
    return r if r.sum() > 0 else p


def verify(rows, drafts, u, v, settings, proposals):
    """One request: rows [n + 1][V], drafts and u [n], proposals a list of (q, q of the draft).

    Returns (accepted, tokens [n + 1] with -1 behind the last, acceptance probabilities [n])."""
    n = len(drafts)
    ps = [shares(z, settings) for z in rows]
    accept = [ratio(ps[i], proposals[i][1], drafts[i])[1] for i in range(n)]
    tokens, k = [-1] * (n + 1), 0
    while k < n and u[k] * proposals[k][1] < ratio(ps[k], proposals[k][1], drafts[k])[0]:
        tokens[k] = drafts[k]
        k += 1
    last = ps[k] if k == n else rest(ps[k], proposals[k][0])
    if last.sum() > 0:
        tokens[k] = sample.draw(last, v)
    return k, tokens, accept
