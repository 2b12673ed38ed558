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


def rising(edit, d, lens):
    """Gives the inputs decays above 1 or a beta outside [0, 2]."""
    import torch
    g, n = d["g"], sum(lens)
    t = torch.arange(n)
    if edit.startswith("beta"):
        b = float(edit[4:])
        d["beta"][:] = b
        g -= math.log(max(1.0, abs(1.0 - b)))   # so that nothing grows
    elif edit == "one small rise":
        g[:] = -0.2
        g[n // 3] = 0.001
    elif edit == "steady rise":
        g[:] = 0.3
    elif edit == "one block's rise":
        g[:] = -0.01
        g[64:128] = 1.0
    elif edit == "up and down":
        g[:] = torch.where(t % 40 < 20, 0.9, -1.1).float()[:, None]
    else:
        assert edit == "one beta"
        d["beta"][n // 2, 1] = 2.5


RISES = ["beta-0.5", "beta-0.01", "beta2.1", "beta2.25", "beta3", "beta-7", "one small rise", "steady rise",
         "one block's rise", "up and down", "one beta"]


@pytest.mark.parametrize("lens", LENS + [[70, 3, 0, 129, 64]], ids=IDS + ["batch"])
@pytest.mark.parametrize("edit", RISES)
def test_decays_above_one_and_any_beta(lens, edit):
    d = inputs(lens, 2, 4, 48, "bf16", 13)
    rising(edit, d, lens)
    hold(d, lens, "bf16")


@pytest.mark.parametrize("dv,act", [(16, "f16"), (128, "bf16"), (256, "bf16")])
def test_rises_at_other_head_sizes(dv, act):
    lens = [200]
    d = inputs(lens, 1, 2, dv, act, 17)
    d["g"][30, 0] = 0.5
    d["beta"][100, 1] = -1.0
    hold(d, lens, act)


@pytest.mark.parametrize("at", [0, 63, 64, 140, 191, 199])
def test_only_the_head_that_rises_is_touched(at):
    # blocks, heads and sequences without a rise keep their results bit for bit
    lens = [200, 100]
    d = inputs(lens, 2, 4, 32, "bf16", 19)
    clean = gpu(d, lens, "bf16")
    d["g"][at, 2] = 0.25
    o, S = gpu(d, lens, "bf16")
    other = [0, 1, 3]
    assert np.array_equal(o[:, other], clean[0][:, other]) and np.array_equal(S[:, other], clean[1][:, other])
    first = at // 64 * 64   # the head's blocks before, and the other sequence
    assert np.array_equal(o[:first, 2], clean[0][:first, 2])
    assert np.array_equal(o[200:], clean[0][200:]) and np.array_equal(S[1], clean[1][1])
    hold(d, lens, "bf16")


def test_rises_in_a_batch_of_many_blocks_as_each_alone():
    # so many blocks that one workgroup may prepare two value heads of a key head
    lens = [25 + 9 * (i % 5) for i in range(50)]
    d = inputs(lens, 16, 64, 16, "bf16", 23)
    d["g"][3::50, ::3] = 0.1
    d["beta"][7::40, 1::5] = 2.2
    got = gpu(d, lens, "bf16")
    at = 0
    for i, n in enumerate(lens):
        if i % 7 == 0:
            one = {k: v[at:at + n] for k, v in d.items() if k != "state"}
            one["state"] = d["state"][i:i + 1]
            alone = gpu(one, [n], "bf16")
            assert np.array_equal(alone[0], got[0][at:at + n]) and np.array_equal(alone[1][0], got[1][i])
        at += n
    hold({k: (v[:1] if k == "state" else v[:lens[0]]) for k, v in d.items()}, lens[:1], "bf16")


def test_captured_with_rises_that_come_and_go():
    import torch
    from int4_routed_expert_router_amd import api
    lens = [150, 40]
    d = inputs(lens, 2, 4, 64, "bf16", 29)
    c = {k: v.cuda() for k, v in d.items()}
    off, s0, n = offsets(lens), c["state"].clone(), sum(lens)
    ws = api.gdn_prefill_workspace(len(lens), n, 2, 4, 64)
    o = [torch.empty(n, 4, 64, device="cuda") for _ in range(2)]
    s = [s0.clone() for _ in range(2)]

    def run(i):
        api.gdn_prefill(c["q"], c["k"], c["v"], c["g"], c["beta"], s[i], o[i], off, Q_SCALE, "bf16", ws=ws)

    run(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(0)
    for at in (None, 20, None, 100, 149):
        c["g"].copy_(d["g"])
        if at is not None:
            c["g"][at] = 0.5
        for x in s:
            x.copy_(s0)
        graph.replay()
        torch.cuda.synchronize()
        run(1)
        torch.cuda.synchronize()
        assert torch.equal(o[0], o[1]) and torch.equal(s[0], s[1])


def uneven(edit, d, lens):
    """Gives the inputs numbers of very different size within a block."""
    import torch
    n = sum(lens)
    gen = torch.Generator().manual_seed(5)
    kind, _, arg = edit.partition(" ")
    if kind == "jump":   # a state far above the values after it
        d["g"][:] = -0.2
        d["g"][n // 2] = 20.0
    elif kind == "large":
        d["g"][:] = -float(arg)
        d["state"] *= 1e6
    elif kind == "novalues":
        d["g"][:] = -float(arg)
        d["v"].zero_()
    elif kind == "values":   # of 10^-5 to 10^5 times their size, by token
        d["v"] = (d["v"].float() * 10 ** (10 * torch.rand(n, 1, 1, generator=gen) - 5)).to(d["v"].dtype)
    elif kind == "betas":
        d["beta"] *= 10 ** (-8 * torch.rand(d["beta"].shape, generator=gen))
    elif kind == "tail":
        d["g"][:] = -0.5
        d["v"][n // 2:] *= 1e-6
    elif kind == "all":
        d["v"] *= float(arg)
        d["state"] *= float(arg)
    else:   # tokens that only decay
        assert kind == "pads"
        d["g"][:] = -5.0
        for e in range(54, n, 32):
            d["v"][e - 10:e] = 0
            d["beta"][e - 10:e] = 0


@pytest.mark.parametrize("lens", LENS + [[70, 3, 129, 64]], ids=IDS + ["batch"])
@pytest.mark.parametrize("edit", ["jump", "large 0.2", "large 0.5", "large 2", "novalues 0.05", "novalues 0.2", "values",
                                  "betas", "tail", "all 1e-34", "all 1e36"])
def test_numbers_of_very_different_size_in_a_block(lens, edit):
    d = inputs(lens, 2, 4, 48, "bf16", 37)
    uneven(edit, d, lens)
    hold(d, lens, "bf16")


@pytest.mark.parametrize("edit", ["novalues 0.5", "novalues 2", "pads"])
def test_what_a_block_shrinks_beyond_its_digits(edit):
    # An operand below 2^-48 of the block's largest counts as zero.  At most 64
    # tokens' products of two such operands, and 64 of one with a key, meet in a
    # result: 2^-40 of the state before the block and of its values on top
    lens = [150]
    d = inputs(lens, 2, 4, 48, "bf16", 37)
    uneven(edit, d, lens)
    got_o, got_s = (x.astype(np.float64) for x in gpu(d, lens, "bf16"))
    o, S, bo, bs = oracle_with_bounds(d, lens)
    size = np.linalg.norm(d["state"].double().numpy()) + np.linalg.norm(d["v"].double().numpy(), axis=-1).max()
    assert (np.linalg.norm(got_o - o, axis=-1) <= bo + 2.0 ** -40 * Q_SCALE * size).all()
    assert (np.sqrt(((got_s - S) ** 2).sum((-1, -2))) <= bs + 2.0 ** -40 * size).all()


@pytest.mark.parametrize("lens", [[9], [24], [90]], ids=["short", "longest short", "blocks"])
def test_overflowing_rows_of_both_kinds_and_large_states(lens):
    # a row whose sum of squares overflows counts as zero, also where the other
    # row of its token, or the state, is large; finite rows up to that size are
    # normalised before they meet a large state
    d = inputs(lens, 1, 2, 32, "bf16", 31)
    d["state"] *= 100.0
    d["state"][:, 1] *= 1e25
    d["k"][5], d["q"][5] = 1e15, -1e15   # not overflowing
    d["k"][6, 0, ::2] = 3e18
    zero = {k: v.clone() for k, v in d.items()}
    for t, k, q in ((1, 1e25, 1e25), (2, 3e38, 10.0), (3, 10.0, 3e38), (7, -3e38, 3e38)):
        for key, x in (("k", k), ("q", q)):
            d[key][t] = zero[key][t] = x
            if abs(x) > 1e19:
                zero[key][t] = 0
    zero["k"][6] = 0   # 64 x 9e36 is above fp32's largest number
    d["k"][8, 0, 0] = zero["k"][8, 0, 0] = 3e38   # one element alone
    zero["k"][8] = 0
    hold(d, lens, "bf16", want=zero)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("size", [1e6, 1e15, 1e30])
def test_large_states_that_decay_past_fp32s_smallest_number(size, act):
    # e^G of a block passes 2^-126 after 4 to 60 tokens, in another token for
    # every head; rows without values, which then have no other size to go by.
    # The floor is that of test_what_a_block_shrinks_beyond_its_digits
    import torch
    lens = [150, 65]
    d = inputs(lens, 1, 16, 48, act, 43)
    d["state"] *= size
    d["v"][..., ::3] = 0
    d["g"][:] = -87.4 / torch.linspace(4.0, 60.0, 16)
    d["g"][:, ::5] -= 0.05 * d["beta"][:, ::5]
    d["beta"][:, 3] *= 1e-20
    d["beta"][:, 4] = 1e-40
    got_o, got_s = (x.astype(np.float64) for x in gpu(d, lens, act))
    o, S, bo, bs = oracle_with_bounds(d, lens)
    assert np.isfinite(got_o).all() and np.isfinite(got_s).all()
    floor = 2.0 ** -40 * np.linalg.norm(d["state"].double().numpy(), axis=(-1, -2)).max()
    assert (np.linalg.norm(got_o - o, axis=-1) <= bo + Q_SCALE * floor).all()
    assert (np.sqrt(((got_s - S) ** 2).sum((-1, -2))) <= bs + floor).all()
