"""Dense product with int4 affine group-quantised weights in float64 (TEST
INFRASTRUCTURE ONLY): y[t, n] = sum_k x[t, k] (s[n, k // G] q[n, k] + b[n, k // G]),
and a bound on the error of fp32 sums of it.
"""
from __future__ import annotations

import numpy as np


def unpack_words(words) -> np.ndarray:
    """[N, K/8] 32-bit words, value 8 i + j in bits 4 j of word i -> [N, K]."""
    w = np.asarray(words).view(np.uint32).astype(np.uint64)
    return np.stack([(w >> np.uint64(4 * j)) & np.uint64(15) for j in range(8)], -1).reshape(w.shape[0], -1).astype(
        np.float64)


def pack_words(q) -> np.ndarray:
    q = np.asarray(q, np.uint32)
    out = np.zeros((q.shape[0], q.shape[1] // 8), np.uint32)
    for j in range(8):
        out |= q[:, j::8] << np.uint32(4 * j)
    return out.view(np.int32)


def linear(x, q, s, b, group: int) -> np.ndarray:
    w = np.repeat(np.asarray(s, np.float64), group, 1) * q + np.repeat(np.asarray(b, np.float64), group, 1)
    return np.asarray(x, np.float64) @ w.T


def error_bound(x, q, s, b, group: int) -> np.ndarray:
    """Bound on |fp32 result - exact| per output, for sums formed as
    16 s (sum (1 + q/16) x) + (b - 16 s) (sum x) per group: every sum of n
    terms, in any order and with each addition off by at most one unit in the
    last place (2^-23), is off by at most n 2^-23 times the sum of the terms'
    magnitudes.  At most 128 terms meet in a group's sums, two additions per
    group (or per 64 columns) and 16 joins follow, and 16 s, b - 16 s round once
    each."""
    ax = np.abs(np.asarray(x, np.float64))
    T, K = ax.shape
    s16 = 16.0 * np.abs(np.asarray(s, np.float64))
    c = np.abs(np.asarray(b, np.float64) - 16.0 * np.asarray(s, np.float64))
    w = np.repeat(s16, group, 1) * (1.0 + q / 16.0) + np.repeat(c, group, 1)
    n = 128 + 2 * (K // min(group, 64)) + 16 + 2
    return n * 2.0 ** -23 * (ax @ w.T)
