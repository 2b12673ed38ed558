"""GPU scored expert choice (moe_select, moe_route_scored) against the fp64
oracle.  Indices must be equal: the kernel orders by keys that agree with the
64-bit ones.  Weights: one rounding of a 64-bit value to fp32 is off by at
most 2^-24 of it; 1% on top covers the 64-bit arithmetic."""
import math

import numpy as np
import pytest

from oracle import moe_oracle as mo
from oracle import select_oracle as so

pytestmark = pytest.mark.gpu

W_TOL = 1.01 * 2.0 ** -24


def run(z, k, kind, bias=None, gate=False, **kw):
    import torch
    from int4_routed_expert_router_amd import api
    z = np.ascontiguousarray(z, np.float32)
    T, E = z.shape
    E -= gate
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    g = torch.full((T,), float("nan"), device="cuda") if gate else None
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    api.select(api.SelectDesc(E, k, kind, **kw), torch.from_numpy(z).cuda(), idx, w, bias=b, shared_gate=g)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy(), None if g is None else g.cpu().numpy()


def check(z, k, kind, bias=None, **kw):
    z = np.asarray(z, np.float32)
    idx, w, _ = run(z, k, kind, bias, **kw)
    ref_i, ref_w = so.select(z, k, kind, None if bias is None else np.asarray(bias, np.float32), **kw)
    bad = np.argwhere((idx != ref_i).any(-1)).ravel()
    assert bad.size == 0, f"tokens {bad[:4].tolist()}: {idx[bad[:1]].tolist()} != {ref_i[bad[:1]].tolist()}"
    assert (np.abs(w - ref_w) <= W_TOL * np.abs(ref_w) + 1e-37).all()
    # the same rows many times over: long batches run on a kernel of their own
    reps = -(-2051 // len(z))
    many_i, many_w, _ = run(np.tile(z, (reps, 1)), k, kind, bias, **kw)
    assert np.array_equal(many_i, np.tile(ref_i, (reps, 1)))
    ref_many = np.tile(ref_w, (reps, 1))
    assert (np.abs(many_w - ref_many) <= W_TOL * np.abs(ref_many) + 1e-37).all()
    return idx, w


CASES = [  # E, K, T, kind, groups, top_groups, group_top, bias, renorm, scale
    (1, 1, 3, "softmax", 1, 1, 1, False, True, 1.0),
    (2, 2, 5, "sigmoid", 2, 1, 2, True, False, 16.0),
    (64, 64, 9, "sigmoid", 1, 1, 1, True, True, 1.0),
    (60, 5, 40, "sigmoid", 15, 4, 2, True, True, 1.0),
    (128, 16, 60, "softmax", 16, 6, 1, True, False, 1.0),
    (250, 16, 33, "sigmoid", 1, 1, 1, True, False, 2.5),
    (65, 1, 70, "softmax", 13, 2, 2, False, True, 1.0),
    (65, 7, 70, "softmax", 1, 1, 1, True, False, 2.5),
    (64, 3, 33, "softmax", 64, 5, 2, False, True, 1.0),
    (160, 6, 50, "softmax", 8, 3, 1, False, False, 16.0),
    (256, 8, 301, "sigmoid", 8, 4, 2, True, True, 2.5),
    (512, 10, 64, "softmax", 1, 1, 1, False, True, 1.0),
    (510, 64, 11, "sigmoid", 5, 2, 2, True, True, 1.0),
    (1000, 33, 17, "sigmoid", 40, 7, 2, True, True, 1.0),
    (1023, 12, 6, "softmax", 3, 2, 2, True, True, 1.0),
    (1024, 64, 5, "sigmoid", 16, 1, 2, True, False, 1.0),
]
CASES = [c if c[4] == 1 or c[0] // c[4] * c[5] >= c[1] else c[:1] + (c[0] // c[4] * c[5],) + c[2:] for c in CASES]


def _id(c):
    return f"E{c[0]}_K{c[1]}_T{c[2]}_{c[3]}_g{c[4]}x{c[5]}"


@pytest.mark.parametrize("case", CASES, ids=_id)
def test_random(case):
    E, K, T, kind, ng, tg, gt, has_bias, renorm, scale = case
    rng = np.random.default_rng(E * 31 + K)
    bias = 0.3 * rng.standard_normal(E) if has_bias else None
    check(1.5 * rng.standard_normal((T, E)), K, kind, bias, n_group=ng, top_groups=tg, group_top=gt, renorm=renorm,
          scale=scale)


@pytest.mark.parametrize("case", CASES, ids=_id)
def test_heavy_ties_and_masks(case):
    # few distinct logits, many experts off; every third row leaves nothing
    E, K, T, kind, ng, tg, gt, has_bias, renorm, scale = case
    rng = np.random.default_rng(E * 37 + K)
    z = rng.integers(-2, 3, (T, E)).astype(np.float32)
    z[rng.random((T, E)) < 0.4] = -np.inf
    z[rng.random((T, E)) < 0.05] = np.nan
    z[::3] = -np.inf
    bias = rng.integers(-1, 2, E) * 0.25 if has_bias else None
    idx, w = check(z, K, kind, bias, n_group=ng, top_groups=tg, group_top=gt, renorm=renorm, scale=scale)
    assert (idx[::3] == -1).all() and (w[::3] == 0).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1), (8, 3)], ids=["all", "grouped"])
def test_keys_nearer_than_a_rounding(kind, groups):
    # logits one or a few fp32 steps apart, in shuffled order, and a bias that
    # cancels most of the differences of the scores: fp32 keys would tie or swap
    rng = np.random.default_rng(5)
    T, E, K = 64, 256, 12
    base = np.float32(0.7)
    steps = rng.integers(0, 40, (T, E))
    z = (base.view(np.int32) + steps).astype(np.int32).view(np.float32)
    check(z, K, kind, None, n_group=groups[0], top_groups=groups[1], group_top=2)
    bias = (1e-9 * rng.standard_normal(E)).astype(np.float32)
    check(z, K, kind, bias, n_group=groups[0], top_groups=groups[1], group_top=2)
    # score + bias nearly constant
    z1 = rng.standard_normal(E).astype(np.float32)
    s1 = np.array(so._scores([float(v) for v in z1], kind)[0])
    bias = (1.0 - s1).astype(np.float32)
    check(np.tile(z1, (T, 1)), K, kind, bias, n_group=groups[0], top_groups=groups[1], group_top=2)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_group_ranks_of_cancelling_keys(kind):
    # the two best keys of every group nearly cancel, so ranks differ by less
    # than the keys' own rounding; and far-down logits whose scores leave fp32
    rng = np.random.default_rng(6)
    T, G, per = 50, 16, 8
    z = rng.standard_normal((T, G * per)).astype(np.float32)
    bias = np.full((G, per), -3e4, np.float32)
    bias[:, 2] = 1000.0 + np.arange(G) % 3
    bias[:, 5] = -bias[:, 2]
    check(z, 5, kind, bias.ravel(), n_group=G, top_groups=3, group_top=2)
    bias[:, 2], bias[:, 5] = 3e38, -3e38
    check(z, 5, kind, bias.ravel(), n_group=G, top_groups=3, group_top=2)
    bias[:, [2, 5]] = -3.3e38
    check(z, 5, kind, bias.ravel(), n_group=G, top_groups=3, group_top=2)
    check(-95 + 8 * z, 20, kind)
    z[:, 0] = 30.0
    check(-70 + 10 * z, 20, kind, n_group=G, top_groups=3, group_top=2)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_extreme_values(kind):
    big = float(np.finfo(np.float32).max)
    rows = [[-big] * 8, [-big, 0, -big, 1, -big, -big, 2, -big], [big, -big, big, 0, 1, 2, 3, 4],
            [np.inf, 1, np.inf, -np.inf, 0, np.nan, 5, 6], [200.0, 199, 90, 89, 88.5, 40, 39, 38],
            [-200.0, -199, -90, -89, -104, -103, -700, -746], [0.0, -0.0, 0.0, -0.0, 0, 0, 0, 0],
            [1e-40, -1e-40, 0, 1e-45, -1e-45, 0, 0, 1e-38]]
    for bias in (None, [np.inf, 0, 0.5, -np.inf, np.nan, 0, big, -big]):
        for gt in (1, 2):
            check(rows, 4, kind, bias, renorm=False)
            check(rows, 8, kind, bias)
            check(rows, 2, kind, bias, n_group=4, top_groups=2, group_top=gt)


@pytest.mark.parametrize("T", [37, 3001])
def test_shared_gate_column_and_stride(T):
    rng = np.random.default_rng(9)
    z = rng.standard_normal((T, 101)).astype(np.float32)
    idx, w, g = run(z, 5, "sigmoid", gate=True)
    ref_i, ref_w = so.select(z[:, :100], 5, "sigmoid")
    assert np.array_equal(idx, ref_i)
    np.testing.assert_allclose(g, mo.sigmoid(z[:, 100].astype(np.float64)), rtol=2e-6)


def test_zero_tokens_and_rows_behind_the_last():
    import torch
    from int4_routed_expert_router_amd import api
    d = api.SelectDesc(100, 3)
    idx = torch.full((6, 3), -7, dtype=torch.int32, device="cuda")
    w = torch.full((6, 3), 5.0, device="cuda")
    z = torch.randn(6, 100, device="cuda")
    api.select(d, z[:0], idx[:0], w[:0])
    api.select(d, z[:5], idx[:5], w[:5])
    torch.cuda.synchronize()
    assert (idx[5] == -7).all() and (w[5] == 5).all() and (idx[:5] >= 0).all()


def test_captured_and_on_another_stream():
    import torch
    from int4_routed_expert_router_amd import api
    d = api.SelectDesc(256, 8, "sigmoid", 8, 4, 2)
    z = torch.randn(64, 256, device="cuda")
    bias = 0.1 * torch.randn(256, device="cuda")
    outs = [(torch.empty(64, 8, dtype=torch.int32, device="cuda"), torch.empty(64, 8, device="cuda")) for _ in range(3)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.select(d, z, *outs[0], bias=bias, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.select(d, z, *outs[1], bias=bias)
    for i in range(4):
        z.copy_(torch.randn(64, 256, device="cuda") + i)
        graph.replay()
        api.select(d, z, *outs[2], bias=bias)
        torch.cuda.synchronize()
        assert torch.equal(outs[1][0], outs[2][0]) and torch.equal(outs[1][1], outs[2][1])


@pytest.mark.parametrize("T", [1, 5, 16, 200])
def test_route_scored_feeds_the_experts(T):
    # router logits, choice and expert FFN in one run; the choice equals the
    # oracle's on the logits the call reports, and the FFN the oracle's sum
    # over the chosen experts (index -1 contributes nothing)
    import dataclasses

    import synth
    import torch
    from int4_routed_expert_router_amd import api
    from moe_testlib import DeviceLayer, act_to_f64, assert_close, desc_for
    wl = dataclasses.replace(synth.TINY, n_experts=24, top_k=6)
    dl = DeviceLayer(wl, 0, router_scale=20.0)
    rng = np.random.default_rng(T)
    bias = (0.3 * rng.standard_normal(24)).astype(np.float32)
    bias[:10] = -np.inf   # 14 left, and 3 of 4 groups of 6 hold at least 2 of them
    dl.router_bias = torch.from_numpy(bias).cuda()
    desc, sel = desc_for(wl), api.SelectDesc(24, 6, "sigmoid", 4, 1, 2, True, 2.5)
    x = torch.from_numpy(synth.tokens(wl, n_tokens=T, seed=77).view(np.int16).copy()).cuda()
    idx = torch.empty(T, 6, dtype=torch.int32, device="cuda")
    w, gam = torch.empty(T, 6, device="cuda"), torch.empty(T, device="cuda")
    logits, y = torch.empty(T, 25, device="cuda"), torch.empty(T, wl.hidden, device="cuda")
    api.route_scored(desc, sel, dl.api_layer(), x, idx, w, gam, logits)
    api.expert_ffn(desc, dl.api_layer(), x, idx, w, gam, y)
    torch.cuda.synchronize()
    z = logits.cpu().numpy()
    x64 = act_to_f64(x, wl.act_dtype)
    z64, zs = mo.router_logits(x64, dl.router_f64(), None)
    assert np.abs(z[:, :24] - z64).max() <= 1e-5 * np.abs(z64).max()
    ref_i, ref_w = so.select(z[:, :24], 6, "sigmoid", bias, n_group=4, top_groups=1, group_top=2, scale=2.5)
    assert np.array_equal(idx.cpu().numpy(), ref_i)
    assert (np.abs(w.cpu().numpy() - ref_w) <= W_TOL * np.abs(ref_w)).all()
    gate = 1 / (1 + np.exp(-z[:, 24].astype(np.float64)))
    np.testing.assert_allclose(gam.cpu().numpy(), gate, rtol=2e-6)

    def ffn(ex, row):
        return mo.expert_ffn(row, ex.wg, ex.wu, ex.wd)

    ref_y = np.zeros((T, wl.hidden))
    for t in range(T):
        for e, we in zip(ref_i[t], ref_w[t]):
            if e >= 0:
                ref_y[t] += we * ffn(dl.oracle_expert(int(e)), x64[t])
        ref_y[t] += gate[t] * ffn(dl.oracle_shared(), x64[t])
    assert_close(y.cpu().numpy(), ref_y, f"T={T}")
