"""GPU Gated DeltaNet over sequences (moe_gdn_prefill) outside the ranges that a
trained layer stays in: decays above 1, beta outside [0, 2], cleared states,
rows whose squares overflow.  Short sequences go token by token and long ones in
blocks, and both are held to the fp64 oracle.

Tolerance, before any run.  A token multiplies an error of the state by at most
a = exp(g) and m = max(1, |1 - beta|) (the norm of I - beta k^ k^T), and adds
roundings of its own: a few dozen fp32 operations on numbers of the size of
a |S|, |beta| a |S| and |beta| |v|, with random signs, for which 8 x 2^-24 of
those is allowed as in the tests of ordinary inputs; the decay itself is off by
2^-24 of its exponent, |g| log2(e).  So with errors of different tokens added in
squares
  e^2 <- (a m e)^2 + (c_g a |S| + c |beta| (a |S| + |v|))^2,   c = 8 x 2^-24,  c_g = c + 1.5 x 2^-24 |g|,
in the Frobenius norm of a head's state, and an output row is off by at most
q_scale (e + c |S|)."""
import math

import numpy as np
import pytest

from oracle import deltanet_oracle as dn
from test_gpu_gdn_prefill import gpu, inputs, offsets

pytestmark = pytest.mark.gpu

C0 = 8 * 2.0 ** -24
Q_SCALE = 128 ** -0.5


def oracle_with_bounds(d, lens):
    """(o, state, bound of o [N, Hv], bound of state [B, Hv]) of the formula in fp64."""
    f = {k: v.double().numpy() for k, v in d.items()}
    S, N, Hv = f["state"].copy(), f["v"].shape[0], f["v"].shape[1]
    o, bo, bs = np.zeros_like(f["v"]), np.zeros((N, Hv)), np.zeros((len(lens), Hv))
    frob = lambda x: np.sqrt((x * x).sum((-1, -2)))  # noqa: E731
    t = 0
    for b, n in enumerate(lens):
        e = np.zeros(Hv)
        for _ in range(n):
            a, beta = np.exp(f["g"][t]), np.abs(f["beta"][t])
            old, v = a * frob(S[b]), np.linalg.norm(f["v"][t], axis=-1)
            c_g = C0 + 1.5 * 2.0 ** -24 * np.where(np.isfinite(f["g"][t]), np.abs(f["g"][t]), 0.0)
            S[b:b + 1], o[t:t + 1] = dn.gdn_step(S[b:b + 1], f["q"][t:t + 1], f["k"][t:t + 1], f["v"][t:t + 1],
                                                 f["g"][t:t + 1], f["beta"][t:t + 1], Q_SCALE)
            m = np.maximum(1.0, np.abs(1.0 - f["beta"][t]))
            e = np.sqrt((a * m * e) ** 2 + (c_g * old + C0 * beta * (old + v)) ** 2)
            bo[t] = Q_SCALE * (e + C0 * frob(S[b]))
            t += 1
        bs[b] = e
    return o, S, bo, bs


def hold(d, lens, act, want=None):
    got_o, got_s = (x.astype(np.float64) for x in gpu(d, lens, act))
    o, S, bo, bs = oracle_with_bounds(d if want is None else want, lens)
    assert np.isfinite(got_o).all() and np.isfinite(got_s).all()
    err_o = np.linalg.norm(got_o - o, axis=-1)
    err_s = np.sqrt(((got_s - S) ** 2).sum((-1, -2)))
    # 2^-149: below fp32's last step
    worst_o, worst_s = (err_o / (bo + 2.0 ** -149)).max(), (err_s / (bs + 2.0 ** -149)).max()
    assert worst_o <= 1 and worst_s <= 1, f"{worst_o:.3g} (o) and {worst_s:.3g} (state) of the bound"


LENS = [[23], [150]]
IDS = ["short", "blocks"]


@pytest.mark.parametrize("lens", LENS, ids=IDS)
@pytest.mark.parametrize("size", [30.0, 3e4, 1e30])
@pytest.mark.parametrize("g0", [-100.0, -float("inf")])
def test_cleared_large_states_are_zero_not_nan(lens, size, g0):
    # every decay of a block is 0, and some state rows get no value: those are 0
    d = inputs(lens, 2, 4, 48, "bf16", 3)
    d["state"] *= size
    d["g"][0] = g0
    d["g"][64:65] = g0
    d["v"][..., ::3] = 0
    hold(d, lens, "bf16")
