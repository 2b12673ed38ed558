"""Scored, biased and group-limited expert choice in float64 (TEST
INFRASTRUCTURE ONLY).

Scores are the softmax or the sigmoid of the logits; a balance bias is added
for the choice alone; with groups, only the experts of the best groups (rank =
sum of the group's best keys) take part; the weights are the chosen experts'
scores, renormalised or not, times a scale.  A logit or key of -inf or NaN
puts an expert off: it is never chosen, and ranks without an expert carry
index -1 and weight 0.  Ties go to the lower group and the lower expert.

Written token by token with Python's own sort, apart from the kernel's and
from any vectorised form.
"""
from __future__ import annotations

import math

import numpy as np


def _scores(z, kind):
    live = [e for e, v in enumerate(z) if not math.isnan(v) and v != -math.inf]
    s = [0.0] * len(z)
    if kind == "sigmoid":
        for e in live:
            # 1 / (1 + exp(-z)) with exp's overflow as its limit
            s[e] = 0.0 if -z[e] > 709.0 else 1.0 / (1.0 + math.exp(-z[e]))
    elif kind == "softmax":
        if live:
            m = max(z[e] for e in live)
            ex = {e: 1.0 if z[e] == m else math.exp(z[e] - m) for e in live}
            tot = math.fsum(ex.values())
            for e in live:
                s[e] = ex[e] / tot
    else:
        raise ValueError(kind)
    return s, live


def select_token(z, k, kind, bias=None, n_group=1, top_groups=0, group_top=1, renorm=True, scale=1.0):
    z = [float(v) for v in z]
    E = len(z)
    s, live = _scores(z, kind)
    key = {}
    for e in live:
        v = s[e] + (0.0 if bias is None else float(bias[e]))
        if not math.isnan(v) and v != -math.inf:
            key[e] = v
    per = E // n_group
    top_groups = top_groups or n_group
    if top_groups < n_group:
        rank = []
        for g in range(n_group):
            best = sorted((key[e] for e in range(g * per, (g + 1) * per) if e in key), reverse=True)[:group_top]
            rank.append(math.fsum(best) if best else -math.inf)
        chosen = sorted(range(n_group), key=lambda g: (-rank[g], g))[:top_groups]
        key = {e: v for e, v in key.items() if e // per in chosen}
    order = sorted(key, key=lambda e: (-key[e], e))[:k]
    w = [s[e] for e in order]
    if renorm:
        tot = math.fsum(w)
        w = [v / tot if tot > 0 else 0.0 for v in w]
    pad = k - len(order)
    return order + [-1] * pad, [scale * v for v in w] + [0.0] * pad


def select(z, k, kind, bias=None, **kw):
    """z [T, E] -> (idx [T, k] int64, w [T, k] float64)."""
    rows = [select_token(r, k, kind, bias, **kw) for r in np.asarray(z, np.float64)]
    return (np.array([r[0] for r in rows], np.int64).reshape(-1, k),
            np.array([r[1] for r in rows], np.float64).reshape(-1, k))
