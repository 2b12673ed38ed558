"""GPU paged attention: the append's form for many tokens and its look-up of many sequences, the causal schedule whose
units are whole, and the decode kernel's weights at their own precision."""
import os
import re

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def case(*a, **k):
    from attn_testlib import Case
    return Case(*a, **k)


# ------------------------------------------------------------------ append
def spread(B, N, rng, rows_before=0):
    """Tokens of B sequences, N in all: none in the first, the last and every third between, where B allows it."""
    new = np.zeros(B, np.int64)
    take = [b for b in range(B) if b not in (0, B - 1) and b % 3] if B > 3 else list(range(B))
    for b in rng.choice(take, N):
        new[b] += 1
    return new, np.concatenate([[0], np.cumsum(new)]) + rows_before


def run_append(hq, hk, d, page, rot, norms, act, B, N, seed, with_q=True, in_place=False):
    import torch
    from int4_routed_expert_router_amd import api
    from oracle import attention_oracle as ao
    from test_gpu_attn import append_inputs, close
    rng = np.random.default_rng(seed)
    new, off = spread(B, N - 5, rng, rows_before=2)          # two rows before the first sequence, three behind the last
    total = new + rng.integers(0, 3 * page, B)
    short = rng.random(B) < 0.1                              # more new tokens than positions
    total[short] = np.maximum(total[short] // 4, 0)
    width = int(total.max()) // page + 2
    table = np.full((B, width), -1, np.int32)
    n_pages = 0
    for b in range(B):
        for p in sorted({x // page for x in range(max(int(total[b] - new[b]), 0), int(total[b]))}):
            table[b, p] = n_pages
            n_pages += 1
    order = rng.permutation(n_pages + 2)
    table = np.where(table >= 0, order[table], -1).astype(np.int32)
    for b in rng.choice(B, max(B // 20, 1)):                 # a page that is none
        table[b, int(total[b]) // page] = n_pages + 2
    q, k, v, qn, kn, freq = append_inputs(hq, hk, d, N, rot, norms, act, seed)
    if norms:
        kn = kn * 1.5
    kc = torch.randn(n_pages + 2, hk, page, d, device="cuda").to(q.dtype)
    vc = torch.randn(n_pages + 2, hk, page, d, device="cuda").to(q.dtype)
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    ref = ao.append(f(kc), f(vc), table, total, off, f(k), f(v), f(q) if with_q else None, f(qn), f(kn), 1e-6, f(freq))
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    before = kc.clone()
    cache = api.KVCache(kc, vc, up(table), up(total))
    if in_place:
        q = q.contiguous()
    was = q.clone()
    qo = q if in_place else torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    api.kv_append(cache, k, v, seq_off=up(off), q=q if with_q else None, q_out=qo if with_q else None,
                  q_norm=qn if with_q else None, k_norm=kn, freq=freq)
    if with_q:
        left = np.isnan(ref[0])
        kept = f(was if in_place else torch.full_like(was, 7.0))
        got = f(qo)
        assert np.array_equal(got[left], kept[left])
        close(np.where(left, 0, got), np.where(left, 0, ref[0]), act)
    close(f(kc), ref[1], act)
    assert np.array_equal(f(vc), ref[2])
    untouched = torch.from_numpy((ref[1] == f(before)).all(-1)).cuda()
    assert torch.equal(kc[untouched], before[untouched])


@pytest.mark.parametrize("hq,hk,d", [
    (40, 8, 64), (96, 24, 64), (12, 4, 128), (30, 10, 128), (64, 8, 128), (16, 2, 256), (16, 16, 256), (7, 1, 256), (5, 1, 256),
])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("rot_part,norms,act", [(1, True, "bf16"), (4, True, "f16"), (0, True, "bf16"), (2, False, "f16"),
                                                (0, False, "bf16")])
def test_append_of_many_tokens(hq, hk, d, with_q, rot_part, norms, act):
    # heads that fill a workgroup's rows of lanes and heads that do not, queries that end inside a lane's rows
    run_append(hq, hk, d, 32, d // rot_part if rot_part else 0, norms, act, 3, 1030, hq + d, with_q)


@pytest.mark.parametrize("B", [64, 65, 130, 4096, 4097])
@pytest.mark.parametrize("N", [1, 7, 900, 1030])
def test_append_of_many_sequences(B, N):
    run_append(16, 2, 256 if N > 1000 else 64, 16, 32, True, "bf16", B, N + 5, B + N)


@pytest.mark.parametrize("hq,hk,d", [(16, 2, 256), (30, 10, 128), (40, 8, 64)])
@pytest.mark.parametrize("N", [200, 1030])
def test_append_in_place_of_many_tokens(hq, hk, d, N):
    run_append(hq, hk, d, 64, d, True, "bf16", 5, N, 3, in_place=True)


# ------------------------------------------------------------------ the causal kernel's schedules
def is_cut(new, total, hq, hk, d):
    """Whether k_attn_prefill cuts units: where the longest is longer than an even share of the whole."""
    from int4_routed_expert_router_amd import build
    text = open(os.path.join(build.CSRC, "attn_prefill.hip")).read()
    start, rows = (int(re.search(rf"constexpr int {n} = (\d+)", text)[1]) for n in ("kStart", "kRows"))
    runs = re.search(r"kRuns = D == 256 \? (\d+) : (\d+)", text)
    tpb, cost, longest = rows // (hq // hk), 0, 0
    for n, t in zip(new, total):
        ends = [t - n + min((j + 1) * tpb, n) for j in range(-(-n // tpb))]
        cost += hk * sum(e + start for e in ends if e > 0)
        longest = max([longest] + [e for e in ends if e > 0])
    return (longest + start) * int(runs[1] if d == 256 else runs[2]) > cost


def rng_list(seed, n, lo, hi):
    return np.random.default_rng(seed).integers(lo, hi, n).tolist()


WHOLE = [  # heads, d, page, act, new, cached
    ((8, 8), 64, 16, "f16", [20 + i % 3 for i in range(75)], [0] * 75),
    ((8, 8), 64, 16, "bf16", [(0 if i % 4 == 1 else 9) for i in range(120)], rng_list(1, 120, 0, 60)),   # some without tokens
    ((4, 2), 64, 32, "f16", [1 + i % 5 for i in range(330)], rng_list(2, 330, 0, 70)),
    ((4, 4), 64, 64, "bf16", [300] * 80, [0] * 80),                       # two blocks each
    ((16, 4), 128, 64, "bf16", [40 + i % 31 for i in range(150)], [0] * 150),
    ((2, 1), 128, 16, "f16", [0] * 64 + [5] * 600, [10] * 664),
    ((12, 4), 128, 32, "f16", [90] * 110, [100] * 110),                    # two blocks each over a prefix
    ((16, 2), 256, 64, "f16", [100] * 60, [37] * 60),
    ((8, 8), 256, 16, "bf16", [0] + [30] * 40 + [0], [50] * 42),
    ((16, 16), 64, 16, "bf16", [3] * 64, [0] * 64),
    ((13, 1), 256, 64, "bf16", [19] * 320, [0] * 320),                     # 19 tokens of 13 heads: 247 rows
]


@pytest.mark.parametrize("heads,d,page,act,new,old", WHOLE, ids=range(len(WHOLE)))
@pytest.mark.parametrize("gate", [True, False])
def test_whole_units(heads, d, page, act, new, old, gate):
    import torch
    total = [a + b for a, b in zip(new, old)]
    assert not is_cut(new, total, *heads, d)
    c = case(new, total, *heads, d, page, act, gate=gate, seed=40)
    o = c.run()
    c.check(o)
    assert torch.equal(o, c.run())


@pytest.mark.parametrize("heads,d,n", [((16, 2), 256, 45), ((8, 8), 64, 75), ((16, 4), 128, 70), ((12, 4), 64, 90)])
@pytest.mark.parametrize("gate", [True, False])
def test_whole_units_of_more_tokens_than_positions(heads, d, n, gate):
    # blocks that see nothing, and blocks of which only the last tokens do
    import torch
    new = [300] * n
    total = [(260, 300, 41, 0, 7)[i % 5] + (0 if i % 3 else 9) for i in range(n)]
    assert not is_cut(new, total, *heads, d)
    c = case(new, total, *heads, d, 64, "bf16", gate=gate, seed=41)
    o = c.run()
    c.check(o)
    for b in range(n):
        first = sum(new[:b])
        assert not o[first : first + new[b] - total[b]].any()
    assert torch.equal(o, c.run())


def test_the_schedules_on_both_sides():
    # the same sequences: whole units, and cut ones beside one that is longer than an even share
    import torch
    new, old = [24] * 90 + [1], [0] * 90 + [20000]
    total = [a + b for a, b in zip(new, old)]
    assert not is_cut(new[:90], total[:90], 8, 8, 64) and is_cut(new, total, 8, 8, 64)
    c = case(new, total, 8, 8, 64, 64, "f16", gate=True, seed=42)
    o = c.run()
    c.check(o)
    from int4_routed_expert_router_amd import api
    p = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
    api.attn_prefill(api.KVCache(c.k, c.v, c.table[:90].contiguous(), c.length[:90].contiguous()), c.q, p,
                     c.off[:91].contiguous(), c.scale, gate=c.gate)
    n = sum(new[:90])
    assert (p[n:] == 7).all()
    p[n:] = o[n:]
    c.check(p)


# ------------------------------------------------------------------ decode's weights
# Held as high + low, both rounded to the type: the low part, at most half a step of the high one, is off by half a step of
# itself, 2^-16 (bf16) and 2^-22 (fp16) of the weight.
WEIGHT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22}


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(16, 2, 256, 64), (8, 8, 64, 16), (12, 4, 128, 32), (5, 1, 64, 256)], ids=str)
def test_decode_of_ragged_batches_at_its_own_precision(shape, act):
    total = [1, 0, 15, 16, 17, 33, 127, 129, 257, 1000, 2049, 5000]
    c = case([1] * len(total), total, *shape, act, gate=shape[0] % 2 == 0, seed=50)
    c.weight_step = WEIGHT[act]
    c.check(c.run(decode=True), decode=True)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (256, 64)])
@pytest.mark.parametrize("n", [2, 16, 32, 50, 64])
def test_decode_weights_are_held_to_more_than_the_type(act, d, page, n):
    """Two weights, 1 and 0.75 + w, on values -0.75 and 1 in turn.  w is three eighths of the type's steps there, so that it
    is what rounding the weight to the type loses: the result, w / 1.75, would be 0 (bf16 8.4e-4, fp16 1.0e-4, against an
    allowed error of 4.9e-5 and 3.3e-5 at 64 positions of 256)."""
    import torch
    from attn_testlib import STEP
    c = case([1] * 2, [n, n], 4, 2, d, page, act, seed=51)
    c.weight_step = WEIGHT[act]
    c.q[:] = 0
    c.q[:, :, 3] = 1.0
    c.scale = float(np.float32(np.log(0.75 + 0.375 * STEP[act])))
    for b in range(2):
        pos = torch.arange(n, device="cuda")
        pages = c.table[b, (pos // page).cpu().tolist()].long()
        c.k[pages, :, pos % page] = 0
        odd = (pos % 2).to(c.k.dtype)
        c.k[pages, :, pos % page, 3] = odd[:, None]
        c.v[pages, :, pos % page] = torch.where(odd > 0, 1.0, -0.75).to(c.v.dtype)[:, None, None]
    c.check(c.run(decode=True), decode=True)


# ------------------------------------------------------------------ the largest calls
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("B", [5000, 65535])
def test_attention_of_the_largest_batches(decode, B):
    # most places of the batch hold nothing
    rng = np.random.default_rng(B)
    live = np.sort(rng.choice(B, 200, replace=False))
    live[0], live[-1] = 0, B - 1
    total = np.zeros(B, np.int64)
    total[live] = rng.integers(1, 40, 200)
    new = np.ones(B, np.int64) if decode else np.zeros(B, np.int64)
    if not decode:
        new[live] = rng.integers(1, 5, 200)              # some with more than they have positions
    c = case(new.tolist(), total.tolist(), 2, 1, 64, 16, "f16", gate=True, seed=60)
    c.check(c.run(decode), decode)


def test_causal_attention_of_the_most_tokens():
    # 2^20 rows, 65535 sequences of 16 that share a page: each sequence's rows are the first one's, up to the last bits
    import torch
    from attn_testlib import STEP
    from int4_routed_expert_router_amd import api
    c = case([16], [16], 2, 1, 64, 16, "bf16", seed=61)
    one = c.run()
    c.check(one)
    B, N = 65535, 1 << 20
    q = c.q[:16].repeat(N // 16, 1, 1)
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    table = c.table[:, :1].repeat(B, 1).contiguous()
    off = torch.arange(B + 1, dtype=torch.int32, device="cuda") * 16
    api.attn_prefill(api.KVCache(c.k, c.v, table, torch.full((B,), 16, dtype=torch.int32, device="cuda")), q, o, off, c.scale)
    want = one[:16].double()
    got = o[: 16 * B].view(B, 16, 2, 64)
    big = c.v[c.table[0, 0].long()].double().abs().max()
    # two results within a rounding of the output and of the weights of the same value each
    assert (got - want).abs().amax(0).le(2 * STEP["bf16"] * (want.abs() + big) + 2.0 ** -14).all()
    assert (o[16 * B :] == 7).all()


@pytest.mark.parametrize("B", [1100, 65535])
def test_append_of_one_token_each(B):
    # no offsets: the form for many tokens, and its twin with offsets
    import torch
    from int4_routed_expert_router_amd import api
    from test_gpu_attn import append_inputs
    hq, hk, d, page = (16, 2, 256, 16) if B < 2000 else (40, 8, 64, 16)
    q, k, v, qn, kn, freq = append_inputs(hq, hk, d, B, d // 2, True, "bf16", 62)
    table = torch.randperm(B, device="cuda").int().view(B, 1)
    length = torch.randint(0, 17, (B,), device="cuda").int()         # 0: no place
    outs = []
    for off in (None, torch.arange(B + 1, dtype=torch.int32, device="cuda")):
        kc = torch.zeros(B, hk, page, d, dtype=q.dtype, device="cuda")
        vc, qo = torch.zeros_like(kc), torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        api.kv_append(api.KVCache(kc, vc, table, length), k, v, seq_off=off, q=q, q_out=qo, q_norm=qn, k_norm=kn, freq=freq)
        outs.append((qo, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    qo, kc, vc = outs[0]
    here = length > 0
    assert (qo[~here] == 7).all() and (qo[here] != 7).any()
    assert torch.equal(vc[table[here, 0].long(), :, (length[here] - 1).long()], v[here])
    assert int((vc != 0).any(-1).any(1).sum()) == int(here.sum())
    # against a sequence at a time, where the other form is taken
    for b in torch.nonzero(here)[:: max(B // 20, 1), 0].tolist():
        k1, v1 = torch.zeros_like(kc[:1]), torch.zeros_like(kc[:1])
        q1 = torch.empty(1, hq, d, dtype=q.dtype, device="cuda")
        api.kv_append(api.KVCache(k1, v1, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), length[b : b + 1]), k[b : b + 1],
                      v[b : b + 1], q=q[b : b + 1], q_out=q1, q_norm=qn, k_norm=kn, freq=freq)
        page_of = int(table[b, 0])
        assert torch.equal(q1[0], qo[b]) and torch.equal(k1[0], kc[page_of]) and torch.equal(v1[0], vc[page_of])


@pytest.mark.parametrize("n", [40, 1100])
def test_append_beyond_32_bits(n):
    # pages whose elements lie beyond 2^32, the same bits as in a small cache
    import torch
    from int4_routed_expert_router_amd import api
    from test_gpu_attn import append_inputs
    hq, hk, d, page = 16, 2, 256, 64
    q, k, v, qn, kn, freq = append_inputs(hq, hk, d, n, 64, True, "bf16", 63)
    m = -(-n // page)
    off, length = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    got = []
    for pages in (m, (1 << 32) // (hk * page * d) + m):
        kc = torch.zeros(pages, hk, page, d, dtype=q.dtype, device="cuda")
        vc = torch.zeros_like(kc)
        table = torch.arange(pages - m, pages, dtype=torch.int32, device="cuda").view(1, m)
        qo = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        api.kv_append(api.KVCache(kc, vc, table, length), k, v, seq_off=off, q=q, q_out=qo, q_norm=qn, k_norm=kn, freq=freq)
        got.append((qo, kc[pages - m :].clone(), vc[pages - m :].clone()))
        assert not kc[: pages - m].any()
        del kc, vc
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("decode", [True, False])
def test_rows_beyond_32_bits(decode):
    # tokens 2^30 elements apart
    import torch
    from int4_routed_expert_router_amd import api
    n, hq, hk, d = 4, 4, 2, 64
    c = case([1] * n if decode else [n], [30, 7, 64, 21] if decode else [90], hq, hk, d, 16, "f16", gate=True, seed=64)
    want = c.run(decode)
    c.check(want, decode)
    step = (1 << 30) + 8
    wide = torch.zeros(3 * step + (2 * hq + 2 * hk) * d, dtype=torch.float16, device="cuda")

    def far(t, at):
        view = wide.as_strided((n, t.shape[1], d), (step, d, 1), at)
        view.copy_(t[:n])
        return view

    q, gate = far(c.q, 0), far(c.gate, hq * d)
    o = torch.full((n, hq, d), 7.0, dtype=torch.float16, device="cuda")
    if decode:
        api.attn_decode(c.cache(), q, o, c.scale, gate=gate)
    else:
        api.attn_prefill(c.cache(), q, o, c.off, c.scale, gate=gate)
    assert torch.equal(o, want[:n])
    kv = torch.randn(n, 2 * hk, d, device="cuda").half()
    k, v = far(kv[:, :hk], 2 * hq * d), far(kv[:, hk:], (2 * hq + hk) * d)
    outs = []
    for a, b in ((k, v), (kv[:, :hk], kv[:, hk:])):
        kc, vc = c.k.clone(), c.v.clone()
        api.kv_append(api.KVCache(kc, vc, c.table, c.length), a, b, seq_off=None if decode else c.off)
        outs.append((kc.view(torch.int16), vc.view(torch.int16)))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and not torch.equal(outs[0][1], c.v.view(torch.int16))
