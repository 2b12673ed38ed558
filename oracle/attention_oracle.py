"""Attention over a paged key-value cache in float64 (TEST INFRASTRUCTURE
ONLY): the cache append with norms and rotary positions, causal softmax
attention with grouped heads and gates, and a bound on the error of fp32
arithmetic with 16-bit softmax weights.

The cache is [pages, kv_heads, page, d], table [B, max_pages], length [B]; off
[B+1] gives each sequence's rows, its last positions (None: one row each).
"""
from __future__ import annotations

import numpy as np


def rows_of(length, off, capacity):
    """(row, sequence, position) of every row that a sequence owns."""
    out = []
    for b, n in enumerate(np.clip(np.asarray(length, np.int64), 0, capacity)):
        first, end = (b, b + 1) if off is None else (int(off[b]), int(off[b + 1]))
        out += [(t, b, int(n) - (end - t)) for t in range(first, end)]
    return out


def _head(x, norm, eps, freq, pos):
    x = np.array(x, np.float64)
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(norm, np.float64)
    if freq is not None:
        r = len(freq)
        a = pos * np.asarray(freq, np.float64)
        u, w = x[..., :r].copy(), x[..., r : 2 * r].copy()
        x[..., :r] = u * np.cos(a) - w * np.sin(a)
        x[..., r : 2 * r] = w * np.cos(a) + u * np.sin(a)
    return x


def append(kc, vc, table, length, off, k, v, q=None, q_norm=None, k_norm=None, eps=1e-6, freq=None):
    """The cache after the call and the queries (NaN in rows that are left out), all float64."""
    kc, vc = np.array(kc, np.float64), np.array(vc, np.float64)
    page = kc.shape[2]
    qo = None if q is None else np.full(np.shape(q), np.nan)
    for t, b, p in rows_of(length, off, table.shape[1] * page):
        if p < 0:
            continue
        if q is not None:
            qo[t] = _head(q[t], q_norm, eps, freq, p)
        at = int(table[b, p // page])
        if 0 <= at < kc.shape[0]:
            kc[at, :, p % page] = _head(k[t], k_norm, eps, freq, p)
            vc[at, :, p % page] = v[t]
    return qo, kc, vc


def attend(kc, vc, table, length, off, q, scale, gate=None, weight_step=0.0):
    """(o, bound): rows that no sequence owns are NaN.  bound: how far fp32
    arithmetic may lie from o before its last rounding, with softmax weights that
    are rounded with a relative error of weight_step.

    With every product and addition off by at most 2^-23 of its result (matrix
    instructions may truncate), n positions and d values of a head: a score is
    off by dz = scale d 2^-23 sum |q k|, its scaled form in the exponent by
    another 4 |z| 2^-23 (scaling, difference to the maximum, exponential), so
    that a weight and the sum of weights are off by factors of 1 + 2 dz + ...;
    adding n weighted values and weights gives 2 n 2^-23 of sum w |v|, and
    dividing, joining and gating less than 40 roundings.  Weights that are held
    in 16 bits are further off by weight_step, and by 2^-31 of the largest where
    they leave fp16's range of full precision."""
    kc, vc = np.asarray(kc, np.float64), np.asarray(vc, np.float64)
    page, group, d = kc.shape[2], q.shape[1] // kc.shape[1], q.shape[2]
    o, bound = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    ulp, of = 2.0 ** -23, {}
    for t, b, p in rows_of(length, off, table.shape[1] * page):
        o[t], bound[t] = 0, 0
        if p >= 0:
            of.setdefault(b, []).append((t, p))
    for b, rows in of.items():
        t, p = (np.array(x) for x in zip(*rows))
        pos = np.arange(p.max() + 1)
        at = np.asarray(table[b], np.int64)[pos // page]
        pos, at = (x[(at >= 0) & (at < kc.shape[0])] for x in (pos, at))
        sees = pos <= p[:, None]
        t, sees = t[sees.any(1)], sees[sees.any(1)]
        for h in range(q.shape[1] if len(t) else 0):
            k, v = kc[at, h // group, pos % page], vc[at, h // group, pos % page]
            n = sees.sum(1, keepdims=True)
            # positions that no row of a block sees may hold anything
            for i in range(0, len(t), 256):
                r, m = t[i : i + 256], int(n[i : i + 256].max())
                ok, qh = sees[i : i + 256, :m], np.asarray(q[r, h], np.float64)
                kk, vv = np.where(ok.any(0)[:, None], k[:m], 0), np.where(ok.any(0)[:, None], v[:m], 0)
                with np.errstate(invalid="ignore"):
                    z = np.where(ok, scale * (qh @ kk.T), -np.inf)
                w = np.exp(z - z.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                if not np.isfinite(vv).all():   # a later token's value must not reach an earlier one's sum
                    o[r, h] = [(w[x][ok[x], None] * vv[ok[x]]).sum(0) for x in range(len(r))]
                    continue
                o[r, h] = w @ vv
                seen_z = np.where(ok, np.abs(z), 0).max(1, keepdims=True)
                dz = (abs(scale) * d * ulp * np.where(ok, np.abs(qh) @ np.abs(kk).T, 0)).max(1, keepdims=True) + 4 * ulp * seen_z
                top = np.where(ok[:, :, None].any(0), np.abs(vv), 0).max(0)
                nn = n[i : i + 256]
                bound[r, h] = (w @ np.abs(vv)) * (weight_step + 2 * dz + 2 * nn * ulp + 40 * ulp) + nn * 2.0 ** -31 * w.max(1, keepdims=True) * top
    if gate is not None:
        s = 1 / (1 + np.exp(-np.asarray(gate, np.float64)))
        o, bound = o * s, bound * s
    return o, bound
