"""GPU paged attention at the limits of its contract: rows that see nothing, scores and values near the ends of fp32's
range, scales of 0 and subnormal ones, tiny rows under a norm, sequences that take no part."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def case(*a, **k):
    from attn_testlib import Case
    return Case(*a, **k)


def same_bits(a, b):
    import torch
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_gates_of_rows_that_see_nothing(decode, value):
    # no positions, or pages that are none: 0 whatever the gate is; the other rows do not change
    new, total = ([1] * 4, [200, 0, 90, 40]) if decode else ([9, 0, 30, 40], [200, 0, 90, 33])
    c = case(new, total, 6, 2, 64, 16, "bf16", gate=True, seed=31)
    c.table[2, :] = -1
    none = [1, 2] if decode else list(range(9, 39)) + list(range(39, 46))   # of the last sequence 7 rows lie before it
    want = c.run(decode)
    c.check(want, decode)
    c.gate[none] = value
    o = c.run(decode)
    assert same_bits(o, want) and not o[none].any()


@pytest.mark.parametrize("act,d", [("bf16", 64), ("f16", 128), ("bf16", 256)])
def test_gates_of_rows_before_a_cut_unit(act, d):
    # one query to a key head: 256 tokens to a unit, whose tiles lie in several runs, its first ten rows at no position
    c = case([300], [290], 2, 2, d, 16, act, gate=True, seed=32)
    want = c.run()
    c.check(want)
    c.gate[:10] = float("nan")
    for _ in range(5):
        assert same_bits(c.run(), want)


def between_the_values(c, o, decode, slack):
    """Each output lies between the values that its row sees, up to slack of the largest."""
    import torch
    v, table, off = c.v.double(), c.table.cpu(), c.off.tolist()
    for b, n in enumerate(c.total):
        m = 1 if decode else c.new[b]
        row0 = b if decode else off[b]
        for i in range(m):
            p = n - m + i
            if p < 0:
                continue
            pos = torch.arange(p + 1)
            seen = v[table[b, pos // c.page].long(), :, pos % c.page].repeat_interleave(c.q.shape[1] // v.shape[1], 1)
            big = seen.abs().amax(0)
            x = o[row0 + i].double()
            assert ((x >= seen.amin(0) - slack * big) & (x <= seen.amax(0) + slack * big)).all(), (b, i)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("exponent", range(20, 47, 2))
def test_scores_of_many_digits(act, decode, exponent):
    """Scores of some 2^exponent have no digits left that tell weights apart, but outputs are still means of values: a
    weight's rounding (half a step of the type, and of the output) and below 2^-12 of fp32 sums of 200 terms."""
    from attn_testlib import STEP
    new, total = ([1] * 3, [150, 1, 70]) if decode else ([150, 1, 40], [150, 1, 70])
    c = case(new, total, 4, 2, 64, 16, act, seed=exponent)
    # |q k| is some 2^10 with 64 products of 1.5 each; then the scale
    for form in range(2):
        if form:   # every key of a head the same
            c.k = c.k.clone()
            for b, n in enumerate(total):
                for p in range(n):
                    c.k[c.table[b, p // 16].long(), :, p % 16] = c.k[c.table[b, 0].long(), :, 0]
        c.scale = 2.0 ** (exponent - 4) * (1 + exponent / 64)
        between_the_values(c, c.run(decode), decode, 2 * STEP[act] + 2.0 ** -12)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("step", [1, 2, 3, 8, 16])
def test_large_scores_that_grow_by_single_steps(act, d, step):
    # scores of 127 x 2^20 + 8 j, exact in fp32 (steps of 8); scaled by log2(e) they keep steps of 8
    import torch
    from attn_testlib import STEP
    n = 160
    c = case([n], [n], 2, 1, d, 32, act, seed=step)
    c.scale = 1.0 / 1.44269504
    c.q[:] = 0
    c.q[:, :, :127] = 1024.0
    c.q[:, :, 127] = 8.0
    c.k[:] = 0
    c.k[..., :127] = 1024.0
    pos = torch.arange(n, device="cuda")
    c.k[c.table[0, (pos // 32)].long(), 0, pos % 32, 127] = (pos // 32 * step).to(c.k.dtype)
    between_the_values(c, c.run(), False, 2 * STEP[act] + 2.0 ** -12)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_whose_sum_just_fits(decode, d):
    # 64 values of up to 2^121: their magnitudes add up to less than 2^127.  Scores rise by 5.5 (8 in powers of two).
    n = 64
    c = case([1] if decode else [n], [n], 2, 1, d, 16, "bf16", seed=33)
    sign = 1 - 2 * (c.v.float() < 0).float()
    c.v = (sign * 2.0 ** 121).to(c.v.dtype)
    c.q[:] = 0
    c.q[:, :, 0] = 1.0
    for p in range(n):
        c.k[c.table[0, p // 16].long(), 0, p % 16] = 0
        c.k[c.table[0, p // 16].long(), 0, p % 16, 0] = 0.0 if p < 32 else 5.5
    c.scale = 1.0
    c.check(c.run(decode), decode)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-39, -1e-39, 1e-44, 2.0 ** -127])
def test_scales_of_none_and_subnormal_ones(decode, scale):
    # products of 2^126 times the scale: 0.06 to 0.85
    c = case([1] if decode else [40], [40], 2, 1, 64, 16, "bf16", seed=34)
    c.q[:] = 0
    c.q[:, 0, 3], c.q[:, 1, 5] = 2.0 ** 63, -2.0 ** 62
    for p in range(40):
        k = c.k[c.table[0, p // 16].long(), 0, p % 16]
        k[:] = 0
        k[3] = 2.0 ** 63 * (p % 3 - 1)
        k[5] = 2.0 ** 63 * (p % 5 - 2)
    c.scale = scale
    # a subnormal scale has fewer digits: the float's own value is meant
    c.scale = float(np.float32(scale))
    c.check(c.run(decode), decode)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 1e-30, 1e-20])
@pytest.mark.parametrize("n", [3, 1100])
def test_norms_of_tiny_rows(act, eps, n):
    import torch
    from int4_routed_expert_router_amd import api
    from oracle import attention_oracle as ao
    from test_gpu_attn import append_inputs, close
    hq, hk, d, page = 4, 2, 128, 64
    q, k, v, qn, kn, freq = append_inputs(hq, hk, d, n, d, True, act, 35)
    # from ordinary rows down to the type's smallest numbers (bf16 2^-133, fp16 2^-24)
    low = 120 if act == "bf16" else 14
    size = 2.0 ** -(torch.arange(n * hq, device="cuda").view(n, hq, 1) % 9 * low / 8)
    q = (q.float() * size).to(q.dtype)
    k = (k.float() * size[:, :hk]).to(k.dtype)
    pages = -(-n // page)
    kc = torch.zeros(pages, hk, page, d, dtype=q.dtype, device="cuda")
    vc = torch.zeros_like(kc)
    cache = api.KVCache(kc, vc, torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1),
                        torch.tensor([n], dtype=torch.int32, device="cuda"))
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    qo = torch.empty(n, hq, d, dtype=q.dtype, device="cuda")
    api.kv_append(cache, k, v, seq_off=off, q=q, q_out=qo, q_norm=qn, k_norm=kn, eps=eps, freq=freq)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    e = float(np.float32(eps))
    for i in range(n):
        close(f(qo[i]), ao._head(f(q[i]), f(qn), e, f(freq), i), act)
        close(f(kc[i // page, :, i % page]), ao._head(f(k[i]), f(kn), e, f(freq), i), act)


@pytest.mark.parametrize("heads,d,n", [((16, 2), 256, 40), ((8, 8), 64, 40), ((4, 4), 128, 80)])
def test_a_sequence_without_tokens_changes_nothing(heads, d, n):
    # an even batch with and without a sequence of a long cache that has no new tokens
    import torch
    from int4_routed_expert_router_amd import api
    c = case([300] * n + [0], [300] * n + [20000], *heads, d, 64, "bf16", seed=36)
    with_it = c.run()
    o = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
    api.attn_prefill(api.KVCache(c.k, c.v, c.table[:n].contiguous(), c.length[:n].contiguous()), c.q, o,
                     c.off[: n + 1].contiguous(), c.scale)
    assert torch.equal(with_it, o)
