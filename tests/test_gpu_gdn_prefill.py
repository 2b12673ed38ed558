"""GPU parity of the Gated DeltaNet over whole sequences (moe_gdn_prefill)
against the fp64 oracle, token by token.

Tolerance, before any run: with |I - beta k k^T| <= 1 and decays <= 1 a
rounding made at one token never grows.  An output passes a few dozen fp32
roundings (dot products of 128 terms, sums over the earlier tokens of its
block), each off by at most 2^-24 of the magnitudes added, with random signs:
8 x 2^-24 in the 2-norm of a whole output, and each of the M tokens that the
slowest head still remembers adds as much: 8 x 2^-24 sqrt(M) with M <= 500 is
1.1e-5.  A single element is allowed 20 times its share."""
import math

import numpy as np
import pytest

from oracle import deltanet_oracle as dn

pytestmark = pytest.mark.gpu

NORM_TOL = 8 * 2.0 ** -24 * math.sqrt(500)


def inputs(lens, hk, hv, dv, act, seed, rate=(0.002, 8.0), k_mean=0.3):
    import torch
    g0 = torch.Generator().manual_seed(seed)
    n = sum(lens)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[act]
    r = lambda *s: torch.randn(*s, generator=g0)  # noqa: E731
    rates = torch.exp(math.log(rate[0]) + torch.rand(hv, generator=g0) * math.log(rate[1] / rate[0]))
    return dict(q=r(n, hk, 128).to(dt), k=(r(n, hk, 128) + k_mean).to(dt), v=r(n, hv, dv).to(dt),
                g=-(rates * torch.nn.functional.softplus(r(n, hv))), beta=torch.sigmoid(1.5 * r(n, hv)),
                state=0.3 * r(len(lens), hv, dv, 128))


def offsets(lens, first=0):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + first, dtype=torch.int32, device="cuda")


def gpu(d, lens, act, q_scale=128 ** -0.5, off=None, **kw):
    import torch
    from int4_routed_expert_router_amd import api
    c = {k: v.cuda() for k, v in d.items()}
    n, hv, dv = d["v"].shape
    o = torch.full((n, hv, dv), 9.0, device="cuda")
    api.gdn_prefill(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], o, offsets(lens) if off is None else off,
                    q_scale, act, **kw)
    torch.cuda.synchronize()
    return o.cpu().numpy(), c["state"].cpu().numpy()


def ref(d, lens, q_scale=128 ** -0.5):
    f = {k: v.double().numpy() for k, v in d.items()}
    S, o = dn.gdn_sequences(f["state"], f["q"], f["k"], f["v"], f["g"], f["beta"], q_scale, lens)
    return o, S


def close(got, want, what):
    got, want = got.astype(np.float64), want.astype(np.float64)
    if not want.size:
        return
    assert np.isfinite(got).all(), what
    norm = np.linalg.norm(want)
    err = np.linalg.norm(got - want)
    assert err <= NORM_TOL * norm, f"{what}: relative error {err / norm:.3g}"
    if norm == 0.0:   # and got is zero too, by the line above
        return
    rms = norm / math.sqrt(want.size)
    worst = (np.abs(got - want) / np.maximum(rms, np.abs(want))).max()
    assert worst <= 20 * NORM_TOL, f"{what}: worst element {worst:.3g}"


def check(lens, hk, hv, dv, act, seed, **kw):
    d = inputs(lens, hk, hv, dv, act, seed, **kw)
    got, want = gpu(d, lens, act), ref(d, lens)
    close(got[0], want[0], "o")
    close(got[1], want[1], "state")
    return d, got


CASES = [  # lens, k_heads, v_heads, dv, act
    ([1], 1, 1, 16, "bf16"), ([2], 2, 4, 128, "f16"), ([5], 16, 32, 128, "bf16"), ([15], 1, 2, 48, "f16"),
    ([16], 1, 1, 64, "bf16"), ([17], 2, 2, 32, "bf16"), ([31, 33], 1, 3, 48, "f16"), ([63], 1, 1, 128, "bf16"),
    ([64], 2, 2, 128, "f16"), ([65], 1, 1, 16, "bf16"), ([127, 0, 129], 2, 6, 80, "bf16"),
    ([128, 1, 64, 0, 0, 200], 1, 2, 256, "f16"), ([300], 3, 3, 112, "bf16"), ([0, 0, 7], 1, 1, 16, "f16"),
    ([3] * 70, 1, 2, 32, "bf16"), ([700], 1, 2, 64, "bf16"),
]


@pytest.mark.parametrize("lens,hk,hv,dv,act", CASES, ids=lambda v: str(v) if not isinstance(v, list) else
                         ("%dx%d" % (len(v), v[0]) if len(v) > 8 else "-".join(map(str, v))))
def test_random(lens, hk, hv, dv, act):
    check(lens, hk, hv, dv, act, seed=sum(lens) * 7 + dv)


@pytest.mark.parametrize("lens", [[6], [150]], ids=["short", "blocks"])
@pytest.mark.parametrize("edit", ["no_decay", "reset", "fast", "cleared_now_and_then", "beta0", "beta1", "beta2", "zero_k", "same_k",
                                  "zero_state", "zero_q", "orthogonal"])
def test_special_inputs(lens, edit):
    import torch
    act = "bf16"
    d = inputs(lens, 2, 4, 32, act, 11)
    n = sum(lens)
    if edit == "no_decay":
        d["g"].zero_()
    elif edit == "reset":
        d["g"][:] = -float("inf")
    elif edit == "fast":
        d["g"][:] = -60.0 - d["beta"]
    elif edit == "cleared_now_and_then":
        d["g"][2::5] = -float("inf")
        d["g"][4::7] = -1e30
    elif edit.startswith("beta"):
        d["beta"][:] = float(edit[4:])
    elif edit == "zero_k":
        d["k"][::3] = 0
    elif edit == "same_k":   # the hardest block: every key is the same, nothing decays, beta 1
        d["k"][:] = d["k"][:1]
        d["beta"][:] = 1.0
        d["g"].zero_()
    elif edit == "zero_state":
        d["state"].zero_()
    elif edit == "zero_q":
        d["q"].zero_()
    else:
        d["k"] = torch.eye(128).repeat(2, 1)[:n].unsqueeze(1).expand(-1, 2, -1).contiguous().to(d["k"].dtype)
    got, want = gpu(d, lens, act), ref(d, lens)
    if edit == "zero_q":
        assert (got[0] == 0).all()
    else:
        close(got[0], want[0], edit)
    close(got[1], want[1], edit)


@pytest.mark.parametrize("act,ks,vs,ss", [("bf16", 1e-3, 1e4, 1e3), ("bf16", 1e6, 1e-6, 1e-8), ("f16", 1e-3, 6e3, 1e5),
                                          ("f16", 500.0, 1e-4, 1e-6), ("bf16", 1e15, 1e20, 1e18), ("bf16", 1.0, 1e-25, 1e-25)])
def test_magnitudes(act, ks, vs, ss):
    # keys, values and states far from 1 (keys are normalised, so only the
    # others' scale shows in the results); columns of very different size
    lens = [70, 3]
    d = inputs(lens, 1, 2, 32, act, 5)
    d["k"] = (d["k"].float() * ks).to(d["k"].dtype)
    d["q"] = (d["q"].float() * ks).to(d["q"].dtype)
    d["v"] = (d["v"].float() * vs).to(d["v"].dtype)
    d["state"] = d["state"] * ss
    d["state"][..., ::2] *= 1e-3
    d["v"][..., 1::4] = 0
    d["state"][:, :, 1::4] = 0
    got, want = gpu(d, lens, act), ref(d, lens)
    for dvi in range(32):   # per state row, so a large one hides no small one
        close(got[0][..., dvi], want[0][..., dvi], f"o {dvi}")
        close(got[1][:, :, dvi], want[1][:, :, dvi], f"state {dvi}")


@pytest.mark.parametrize("hk", [16, 64])
def test_many_blocks_as_each_alone(hk):
    # so many blocks that one workgroup prepares two value heads of a key head
    # (with four or one value heads each)
    lens = [25 + 9 * (i % 5) for i in range(50)]
    d, got = check(lens, hk, 64, 16, "bf16", 41)
    at = 0
    for i, n in enumerate(lens):
        if i % 7 == 0:
            one = {k: v[at:at + n] for k, v in d.items() if k != "state"}
            one["state"] = d["state"][i:i + 1]
            alone = gpu(one, [n], "bf16")
            assert np.array_equal(alone[0], got[0][at:at + n]), (i, n)
            assert np.array_equal(alone[1][0], got[1][i]), (i, n)
        at += n


@pytest.mark.parametrize("lens", [[9], [90]], ids=["short", "blocks"])
def test_rows_whose_squares_overflow_count_as_zero(lens):
    d = inputs(lens, 1, 2, 32, "bf16", 31)
    zero = {k: v.clone() for k, v in d.items()}
    for key, rows in (("k", slice(2, None, 7)), ("q", slice(3, None, 5))):
        d[key][rows] = 1e25
        zero[key][rows] = 0
    got, want = gpu(d, lens, "bf16"), ref(zero, lens)
    close(got[0], want[0], "o")
    close(got[1], want[1], "state")


def test_full_size_layer_long_and_ragged():
    # the listed sizes' heads; checked on one key head's value heads at a time
    # would hide the others, so the oracle runs on every head of a shorter batch
    check([130, 1, 0, 67], 16, 32, 128, "bf16", 21)


def test_a_sequences_results_do_not_depend_on_the_batch():
    lens = [70, 5, 0, 129, 64]
    d = inputs(lens, 2, 4, 48, "bf16", 31)
    o, S = gpu(d, lens, "bf16")
    at = np.concatenate([[0], np.cumsum(lens)])
    for b, n in enumerate(lens):
        one = {k: (v[b:b + 1] if k == "state" else v[at[b]:at[b + 1]]).contiguous() for k, v in d.items()}
        if n == 0:
            assert np.array_equal(S[b], d["state"][b].numpy())
            continue
        o1, S1 = gpu(one, [n], "bf16")
        assert np.array_equal(o1, o[at[b]:at[b + 1]]) and np.array_equal(S1[0], S[b])


@pytest.mark.parametrize("dv,act", [(48, "bf16"), (128, "f16")])
def test_many_short_sequences_as_each_alone(dv, act):
    # enough state rows that a lane takes several; lengths around the longest
    # that goes token by token; rows of d_v past the last group of 64
    lens = [(7 * i) % 26 for i in range(24)] + [90]
    d, got = check(lens, 4, 8, dv, act, 23)
    at = 0
    for i, n in enumerate(lens):
        one = {k: v[at:at + n] for k, v in d.items() if k != "state"}
        one["state"] = d["state"][i:i + 1]
        alone = gpu(one, [n], act)
        assert np.array_equal(alone[0], got[0][at:at + n]), (i, n)
        assert np.array_equal(alone[1][0], got[1][i]), (i, n)
        at += n


def test_continues_where_it_stopped_and_agrees_with_the_step():
    import torch
    from int4_routed_expert_router_amd import api
    n = 150
    d = inputs([n], 2, 4, 64, "f16", 41)
    whole_o, whole_s = ref(d, [n])
    c = {k: v.cuda() for k, v in d.items()}
    o = torch.empty(n, 4, 64, device="cuda")
    for a, b in ((0, 64), (64, 65), (65, 140)):
        api.gdn_prefill(c["q"][a:b], c["k"][a:b], c["v"][a:b], c["g"][a:b], c["beta"][a:b], c["state"], o[a:b],
                        offsets([b - a]), 128 ** -0.5, "f16")
    for t in range(140, n):
        api.gdn_step(c["q"][t:t + 1], c["k"][t:t + 1], c["v"][t:t + 1], c["g"][t:t + 1], c["beta"][t:t + 1],
                     c["state"], o[t:t + 1], 128 ** -0.5, "f16")
    torch.cuda.synchronize()
    close(o.cpu().numpy(), whole_o, "o")
    close(c["state"].cpu().numpy(), whole_s, "state")


def test_rows_outside_the_sequences_and_bad_offsets():
    import torch
    lens = [40, 70]
    d = inputs([10] + lens + [13], 1, 2, 32, "bf16", 51)
    d["state"] = d["state"][:2].contiguous()
    inner = {k: (v if k == "state" else v[10:120].contiguous()) for k, v in d.items()}
    for k in ("q", "k", "v", "g", "beta"):
        d[k][:10] = float("nan")
        d[k][120:] = float("inf")
    o, S = gpu(d, None, "bf16", off=offsets(lens, 10))
    close(o[10:120], ref(inner, lens)[0], "o")
    close(S, ref(inner, lens)[1], "state")
    assert (o[:10] == 9.0).all() and (o[120:] == 9.0).all()
    # offsets outside [0, N] are read as its ends; an end before its start as an empty sequence
    n = d["v"].shape[0]
    o, S = gpu(inner, None, "bf16", off=torch.tensor([-5, 40, 2 ** 30], dtype=torch.int32, device="cuda"))
    close(o, ref(inner, lens)[0], "o")
    o, S = gpu(inner, None, "bf16", off=torch.tensor([n + 9, 3, 3], dtype=torch.int32, device="cuda"))
    assert (o == 9.0).all() and np.array_equal(S, inner["state"].numpy())


def test_nonfinite_values_stay_in_their_sequence():
    lens = [70, 66, 5]
    d = inputs(lens, 1, 2, 32, "bf16", 61)
    clean = gpu(d, lens, "bf16")
    d["v"][75], d["k"][80], d["g"][90], d["beta"][100] = float("inf"), float("nan"), float("nan"), float("inf")
    o, S = gpu(d, lens, "bf16")
    for sl in (slice(0, 70), slice(136, 141)):
        assert np.array_equal(o[sl], clean[0][sl])
    assert np.array_equal(S[[0, 2]], clean[1][[0, 2]]) and not np.isfinite(S[1]).all()
    # a non-finite query only reaches its own output
    for bad in ("nan", "inf"):
        d = inputs(lens, 1, 2, 32, "bf16", 61)
        d["q"][76, 0, 5] = float(bad)
        o, S = gpu(d, lens, "bf16")
        keep = np.arange(141) != 76
        assert np.array_equal(o[keep], clean[0][keep]) and np.array_equal(S, clean[1])
        assert bad == "inf" or np.isnan(o[76]).all()


@pytest.mark.parametrize("lens", [[5], [200, 30]], ids=["short", "blocks"])
def test_captured_repeatable_and_on_another_stream(lens):
    import torch
    from int4_routed_expert_router_amd import api
    d = inputs(lens, 2, 4, 64, "bf16", 71)
    c = {k: v.cuda() for k, v in d.items()}
    n = sum(lens)
    off, s0 = offsets(lens), c["state"].clone()

    def run(o, state, **kw):
        api.gdn_prefill(c["q"], c["k"], c["v"], c["g"], c["beta"], state, o, off, 0.1, "bf16", **kw)

    outs = [torch.empty(n, 4, 64, device="cuda") for _ in range(3)]
    states = [s0.clone() for _ in range(3)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    run(outs[0], states[0], stream=st)
    st.synchronize()
    ws = api.gdn_prefill_workspace(len(lens), n, 2, 4, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[2], states[2], ws=ws)
    states[2].copy_(s0)
    for i in range(4):
        run(outs[1], states[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[1], outs[2]) and torch.equal(states[1], states[2])
        if i == 0:
            assert torch.equal(outs[0], outs[1]) and torch.equal(states[0], states[1])
        c["v"].copy_(torch.randn_like(c["v"]))


def test_no_tokens_leave_the_state():
    import torch
    from int4_routed_expert_router_amd import api
    d = inputs([0, 0], 1, 2, 32, "bf16", 81)
    c = {k: v.cuda() for k, v in d.items()}
    s0 = c["state"].clone()
    api.gdn_prefill(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], torch.empty(0, 2, 32, device="cuda"),
                    offsets([0, 0]), 1.0)
    torch.cuda.synchronize()
    assert torch.equal(c["state"], s0)
