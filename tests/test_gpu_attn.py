"""GPU paged attention (moe_kv_append, moe_attn_decode, moe_attn_prefill) against the fp64 oracle."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SHAPES = [  # q heads, kv heads, head dim, page
    (16, 2, 256, 64), (8, 8, 64, 16), (12, 4, 128, 32), (16, 1, 256, 128), (5, 1, 64, 256), (6, 2, 128, 16),
]
shape_ids = ["x".join(map(str, s)) for s in SHAPES]


def case(*a, **k):
    from attn_testlib import Case
    return Case(*a, **k)


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=shape_ids)
def test_decode_of_ragged_batches(shape, act):
    # lengths from none and one, around pages and tiles, to some thousand
    total = [1, 0, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 1000, 2049]
    c = case([1] * len(total), total, *shape, act, gate=shape[0] % 2 == 0, seed=len(act) + shape[0])
    c.check(c.run(decode=True), decode=True)


@pytest.mark.parametrize("length", [1, 2, 3, 64, 500, 4097, 30001])
def test_decode_of_one_sequence(length):
    c = case([1], [length], 16, 2, 256, 64, "bf16", gate=True, seed=length)
    o = c.run(decode=True)
    c.check(o, decode=True)
    import torch
    assert torch.equal(o, c.run(decode=True))


@pytest.mark.parametrize("B", [63, 64, 65, 130, 700])
def test_decode_of_many_sequences(B):
    rng = np.random.default_rng(B)
    total = rng.integers(0, 70, B).tolist()
    c = case([1] * B, total, 4, 2, 64, 16, "f16", seed=B)
    c.check(c.run(decode=True), decode=True)


# ------------------------------------------------------------------ prefill
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=shape_ids)
def test_prefill_of_packed_prompts(shape, act):
    new = [1, 0, 2, 15, 16, 17, 63, 64, 65, 130, 0, 0, 259]
    c = case(new, new, *shape, act, gate=shape[0] % 2 == 0, seed=7 + shape[0])
    c.check(c.run())


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES[:4], ids=shape_ids[:4])
def test_prefill_over_cached_tokens(shape, act):
    new, old = [5, 1, 40, 0, 129, 3], [700, 0, 1, 50, 333, 2000]
    c = case(new, [a + b for a, b in zip(new, old)], *shape, act, gate=shape[0] % 2 == 0, seed=9 + shape[0])
    c.check(c.run())


@pytest.mark.parametrize("new,old", [(1, 0), (1, 5000), (5, 4096), (33, 9000), (300, 1), (1500, 0), (700, 1300)])
def test_prefill_of_one_sequence(new, old):
    import torch
    c = case([new], [new + old], 16, 2, 256, 64, "bf16", gate=True, seed=new)
    o = c.run()
    c.check(o)
    assert torch.equal(o, c.run())


@pytest.mark.parametrize("B", [64, 65, 300])
def test_prefill_of_many_sequences(B):
    rng = np.random.default_rng(B)
    new = rng.integers(0, 6, B)
    total = new + rng.integers(0, 60, B)
    c = case(new.tolist(), total.tolist(), 4, 2, 64, 16, "f16", seed=B)
    c.check(c.run())


@pytest.mark.parametrize("shape,new,old", [
    ((16, 2, 256, 64), [100 + i % 31 for i in range(40)], [0] * 40),        # more units than compute units, none cut
    ((4, 2, 64, 16), [1 + i % 3 for i in range(100)], [3000 if i == 77 else i % 20 for i in range(100)]),
    ((2, 1, 128, 32), [0] * 70 + [400], [9] * 70 + [1000]),                 # the only tokens come last
    ((16, 1, 128, 128), [3, 1], [2500, 0]),
    ((11, 1, 256, 16), [50], [77]), ((7, 1, 64, 16), [90, 1], [3, 500]), ((13, 1, 128, 64), [64], [0]),
], ids=str)
def test_prefill_of_uneven_batches(shape, new, old):
    c = case(new, [a + b for a, b in zip(new, old)], *shape, "bf16", seed=len(new))
    c.check(c.run())


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes(seed):
    # any group up to 16, pages, lengths, both calls on the same cache
    import random
    r = random.Random(seed)
    hk, d, page = r.choice((1, 1, 2, 3)), r.choice((64, 128, 256)), r.choice((16, 32, 64, 128, 256))
    B = r.choice((1, 2, 5, 17, 70))
    most = 1500 // B
    new = [r.choice((0, 1, 1, 2, r.randint(0, 40), r.randint(0, most // 3 + 1))) for _ in range(B)]
    old = [r.choice((0, 1, r.randint(0, most), r.randint(0, 2 * most))) for _ in range(B)]
    c = case(new, [a + b for a, b in zip(new, old)], hk * r.randint(1, 16), hk, d, page, r.choice(("bf16", "f16")),
             gate=r.random() < 0.5, seed=seed, spread=r.choice((0.3, 1.5, 4.0)))
    c.check(c.run())
    if c.q.shape[0] >= B:
        c.check(c.run(decode=True), decode=True)


# ------------------------------------------------------------------ what no token may see
@pytest.mark.parametrize("decode", [True, False])
def test_more_new_tokens_than_positions_and_lengths_out_of_range(decode):
    import torch
    c = case([3, 4, 2, 1], [40, 30, 32, 1], 4, 2, 64, 16, "bf16", width=3)
    # sequence 0: fuller than its table; 1: rows at positions -2, -1, 0, 1; 2: below 0
    c.length = torch.tensor([1000, 2, -5, 1], dtype=torch.int32).cuda()
    c.table[0] = c.table[0].clamp(min=0)
    c.k[c.table[0, 2].long()] = 0.5
    c.v[c.table[0, 2].long()] = 0.5
    o = c.run(decode)
    c.check(o, decode)
    if not decode:
        assert not o[3:5].any() and not o[7:9].any() and o[5].any()
    else:
        assert not o[2].any()


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("page,d", [(16, 64), (64, 256)])
def test_pages_that_are_none(decode, page, d):
    new, total = ([1] * 4, [200, 333, 90, 40]) if decode else ([9, 50, 1, 40], [200, 333, 90, 40])
    c = case(new, total, 4, 2, d, page, "bf16", seed=1)
    n = c.k.shape[0]
    c.table[0, 1], c.table[1, 0], c.table[1, 2] = -1, n, -2 ** 31
    c.table[2, :] = 2 ** 31 - 1                  # nothing left
    c.table[3, -(-40 // page) - 1] = -5          # the newest tokens' page
    o = c.run(decode)
    c.check(o, decode)
    first = 2 if decode else 59
    assert not o[first : first + 1].any()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 6e4])
@pytest.mark.parametrize("act,d", [("bf16", 256), ("f16", 128), ("bf16", 64)])
def test_later_tokens_do_not_reach_earlier_ones(act, d, value):
    import torch
    new, old = [70, 0, 37, 200], [3, 9, 500, 11]
    c = case(new, [a + b for a, b in zip(new, old)], 6, 2, d, 16, act, seed=3)
    clean = c.run()
    c.check(clean)
    own = torch.zeros(c.q.shape[0], dtype=torch.bool)
    for b, at in ((0, 40), (2, 36), (3, 5), (3, 120)):   # rows whose keys and values hold something else
        pos = old[b] + at
        page = c.table[b, pos // 16].long()
        for t in (c.k, c.v):
            t[page, 1, pos % 16, 5 : d : 7] = value
        row = int(c.off[b]) + at
        own[row : int(c.off[b + 1])] = True
    o = c.run()
    assert torch.equal(o[:, :3], clean[:, :3])               # the other key head's
    before = ~own.cuda()
    assert torch.equal(o[before], clean[before])


@pytest.mark.parametrize("decode", [True, False])
def test_scores_of_minus_infinity(decode):
    import torch
    new, total = ([1, 1], [40, 33]) if decode else ([20, 33], [40, 33])
    c = case(new, total, 2, 1, 64, 16, "bf16", seed=5)
    c.q[:, :, 1:] = 0
    c.q[:, :, 0] = 1.0
    c.k[c.table[0, 0].long(), 0, 3, 0] = -float("inf")       # one weight of 0
    for i in range(3):
        c.k[c.table[1, i].long(), :, :, 0] = -float("inf")   # nothing but such
    o = c.run(decode)
    w = 0 if decode else slice(0, 20)
    assert torch.isfinite(o[w].float()).all() and o[w].any()
    assert not o[1 if decode else slice(20, 53)].any()


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_large_scores_and_scales(act, decode):
    # one weight of almost 1 and large differences; equal scores; a negative scale
    new, total = ([1] * 3, [300, 2, 77]) if decode else ([40, 2, 60], [300, 2, 77])
    for scale in (30.0, 0.0, -0.7, 1e-30):
        c = case(new, total, 6, 2, 128, 32, act, gate=True, seed=11)
        c.scale = scale
        c.check(c.run(decode), decode)


@pytest.mark.parametrize("decode", [True, False])
def test_values_of_either_end_of_the_types(decode):
    import torch
    new, total = ([1] * 2, [300, 129]) if decode else ([17, 129], [300, 129])
    for act, big in (("bf16", 2.0 ** 110), ("f16", 2.0 ** 15), ("f16", 2.0 ** -20), ("bf16", 2.0 ** -100)):
        c = case(new, total, 6, 2, 64, 16, act, seed=12)
        c.v = (c.v.float() / 16 * big).to(c.v.dtype)
        c.check(c.run(decode), decode)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ layouts, streams, graphs
@pytest.mark.parametrize("decode", [True, False])
def test_rows_of_other_strides(decode):
    import torch
    new, total = ([1] * 5, [100, 7, 64, 0, 31]) if decode else ([20, 7, 64, 0, 31], [100, 7, 64, 0, 31])
    c = case(new, total, 6, 2, 64, 16, "f16", gate=True, seed=13)
    want = c.run(decode)
    c.check(want, decode)
    q, gate = c.q.clone(), c.gate.clone()
    for form in range(3):
        if form == 0:     # heads first
            c.q, c.gate = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, gate))
        elif form == 1:   # wide rows
            wide = torch.zeros(q.shape[0], 6, 64 + 24, dtype=q.dtype, device="cuda")
            wide[:, :, 8:72] = q
            c.q, c.gate = wide[:, :, 8:72], gate.contiguous()
        else:             # the same row for every token
            c.q, c.gate = q[:1].expand(q.shape), gate[:, :1].expand(gate.shape)
        o = c.run(decode)
        c.check(o, decode)
        if form < 2:
            assert torch.equal(o, want)


def test_shared_pages_and_long_tables():
    # sequences that share a prefix; a table far wider than the lengths
    import torch
    c = case([4, 4, 1], [100, 100, 60], 4, 2, 128, 32, "bf16", width=5000, seed=14)
    c.table[1, :3] = c.table[0, :3]
    c.check(c.run())
    c.check(c.run(decode=True), decode=True)
    torch.cuda.synchronize()


@pytest.mark.parametrize("decode", [True, False])
def test_offsets_beyond_32_bits(decode):
    import torch
    from attn_testlib import Case
    hk, d, page = 2, 256, 64
    n_pages = (1 << 32) // (hk * d * page) + 100          # elements beyond 2^32
    small = Case([1, 9] if decode is False else [1, 1], [500, 777], 8, hk, d, page, "bf16", seed=15)
    want = small.run(decode)
    small.check(want, decode)
    k = torch.zeros(n_pages, hk, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    m = small.k.shape[0]
    at = torch.arange(m, device="cuda") + torch.where(torch.arange(m, device="cuda") % 2 == 0, n_pages - m, 0)
    k[at], v[at] = small.k, small.v
    small.k, small.v = k, v
    small.table = torch.where(small.table < 0, small.table, at.int()[small.table.clamp(min=0).long()]).contiguous()
    assert torch.equal(small.run(decode), want)


@pytest.mark.parametrize("decode", [True, False])
def test_another_stream_and_given_workspaces(decode):
    import torch
    from int4_routed_expert_router_amd import api
    new, total = ([1] * 3, [3000, 5, 700]) if decode else ([100, 5, 7], [3000, 5, 700])
    c = case(new, total, 16, 2, 256, 64, "bf16", gate=True, seed=16)
    want = c.run(decode)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = c.run(decode)
    s.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    b = c.run(decode, stream=s)
    s.synchronize()
    ws = api.attn_workspace(c.cache(), 16, 200)
    ws.fill_(255)
    d = c.run(decode, ws=ws)
    for o in (a, b, d):
        assert torch.equal(o, want)


def test_two_calls_at_once():
    import torch
    cs = [case([1] * 4, [4000, 900, 0, 77], 16, 2, 256, 64, "bf16", seed=20),
          case([500, 30], [900, 4000], 16, 2, 256, 64, "bf16", seed=21)]
    want = [cs[0].run(True), cs[1].run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, c, decode in zip(streams, cs, (True, False)):
            with torch.cuda.stream(s):
                got.append(c.run(decode))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("decode", [True, False])
def test_captured_calls_follow_the_lengths(decode):
    # one graph, replayed while lengths, offsets and tables change under it
    import torch
    from int4_routed_expert_router_amd import api
    new, total = ([1] * 3, [2000, 5, 700]) if decode else ([90, 5, 40], [2000, 5, 700])
    c = case(new, total, 16, 2, 256, 64, "bf16", gate=True, seed=17)
    cache, n = c.cache(), 3 if decode else c.q.shape[0]
    ws = api.attn_workspace(cache, 16, n)
    q, gate = c.q[:n], c.gate[:n]
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")

    def call():
        if decode:
            api.attn_decode(cache, q, o, c.scale, gate=gate, ws=ws)
        else:
            api.attn_prefill(cache, q, o, c.off, c.scale, gate=gate, ws=ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens, offs in (([2000, 5, 700], [0, 90, 95, 135]), ([1, 5, 64], [0, 1, 6, 60]), ([1999, 0, 1], [0, 100, 100, 101]),
                       ([2000, 5, 700], [0, 90, 95, 135])):
        c.length.copy_(torch.tensor(lens, dtype=torch.int32))
        if not decode:
            c.off.copy_(torch.tensor(offs, dtype=torch.int32))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c.check(o, decode)
        assert torch.equal(o, c.run(decode))


def test_two_graphs_that_share_a_workspace():
    import torch
    from int4_routed_expert_router_amd import api
    a = case([1] * 4, [4000, 900, 0, 77], 16, 2, 256, 64, "bf16", seed=20)
    b = case([500, 30], [900, 4000], 16, 2, 256, 64, "bf16", seed=21)
    want = [a.run(True), b.run()]
    ws = api.attn_workspace(b.cache(), 16, 600)
    outs, graphs = [], []
    for c, decode in ((a, True), (b, False)):
        cache, n = c.cache(), len(c.new) if decode else c.q.shape[0]
        o, q = torch.full(c.q[:n].shape, 7.0, dtype=c.q.dtype, device="cuda"), c.q[:n]

        def call():
            if decode:
                api.attn_decode(cache, q, o, c.scale, ws=ws)
            else:
                api.attn_prefill(cache, q, o, c.off, c.scale, ws=ws)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, cache))
        outs.append(o)
    for _ in range(3):
        for o in outs:
            o.fill_(7.0)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
        a.run(True)
        torch.cuda.synchronize()


def test_offsets_in_no_order_stay_within_the_buffers():
    # results are not defined, but every row outside the ranges keeps its values and nothing else is written
    import torch
    from int4_routed_expert_router_amd import api
    c = case([30, 30, 30], [200, 300, 400], 4, 2, 64, 16, "bf16", seed=22)
    n = c.q.shape[0]
    for off in ([50, 10, 60, 20], [-7, 2 ** 31 - 1, -2 ** 31, 5], [92, 92, 0, 0], [0, 1000, 20, 90]):
        c.off = torch.tensor(off, dtype=torch.int32).cuda()
        pad = torch.full((n + 4, 4, 64), 7.0, dtype=c.q.dtype, device="cuda")
        api.attn_prefill(c.cache(), c.q, pad[2 : n + 2], c.off, c.scale)
        k, v = (torch.randn(n, 2, 64, device="cuda").to(c.q.dtype) for _ in range(2))
        kc, vc = c.k.clone(), c.v.clone()
        api.kv_append(api.KVCache(kc, vc, c.table, c.length), k, v, seq_off=c.off)
        torch.cuda.synchronize()
        assert (pad[:2] == 7).all() and (pad[n + 2 :] == 7).all()


# ------------------------------------------------------------------ append
APPENDS = [  # q heads, kv heads, d, page, rot, norms, act
    (16, 2, 256, 64, 64, True, "bf16"), (12, 4, 128, 16, 128, False, "f16"), (8, 8, 64, 32, 16, True, "f16"),
    (3, 3, 256, 128, 256, True, "bf16"), (2, 1, 64, 16, 0, False, "bf16"), (4, 2, 128, 256, 0, True, "bf16"),
    (16, 1, 64, 64, 64, True, "bf16"), (40, 8, 256, 16, 128, False, "f16"),
]


def append_inputs(hq, hk, d, n, rot, norms, act, seed):
    import torch
    from attn_testlib import DT
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rows = r(n, (2 * hq + 2 * hk) * d).to(DT[act]).cuda()
    q = rows[:, : 2 * hq * d].view(n, hq, 2, d)[:, :, 0]
    k, v = rows[:, 2 * hq * d :].view(n, 2, hk, d).unbind(1)
    w = [1 + 0.3 * r(d) if norms else None for _ in range(2)]
    freq = 1e6 ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1)) if rot else None
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    return q, k, v, up(w[0]), up(w[1]), up(freq)


def close(got, ref, act):
    """One rounding to the type after fp32 arithmetic.  A normalised value is off by the sum of d squares (relative
    d 2^-24 / 2 under the root), the root, the division and two products; a rotated one by the angle (fp64, then fp32 at
    up to pi: 2^-22), sine and cosine (2^-22) and three operations: below 256 2^-24 of the largest value of its pair."""
    from attn_testlib import STEP, TINY
    big = np.abs(ref).max(-1, keepdims=True)
    assert (np.abs(got - ref) <= STEP[act] * np.abs(ref) + 2.0 ** -16 * big + TINY[act]).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("hq,hk,d,page,rot,norms,act", APPENDS)
@pytest.mark.parametrize("new,old", [([1], [0]), ([1, 1, 1], [5, 262143, 0]), ([40, 0, 3, 100, 17], [0, 9, 1000, 15, 16])])
def test_append(hq, hk, d, page, rot, norms, act, new, old):
    import torch
    from int4_routed_expert_router_amd import api
    from oracle import attention_oracle as ao
    total = [a + b for a, b in zip(new, old)]
    n, width = sum(new), max(total) // page + 2
    pages = [sorted({p // page for p in range(t - m, t)}) for m, t in zip(new, total)]
    n_pages = sum(map(len, pages)) + 2
    order = torch.randperm(n_pages).tolist()
    table = torch.full((len(new), width), -1, dtype=torch.int32)
    for b, ps in enumerate(pages):
        for p in ps:
            table[b, p] = order.pop()
    q, k, v, qn, kn, freq = append_inputs(hq, hk, d, n + 2, rot, norms, act, n + d)
    kc = torch.randn(n_pages, hk, page, d, device="cuda").to(q.dtype)
    vc = torch.randn(n_pages, hk, page, d, device="cuda").to(q.dtype)
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    off = np.concatenate([[0], np.cumsum(new)])
    ref = ao.append(f(kc), f(vc), table.numpy(), np.array(total), off, f(k), f(v), f(q), f(qn), f(kn), 1e-6, f(freq))
    before = kc.clone(), vc.clone()
    length, offs = torch.tensor(total, dtype=torch.int32).cuda(), torch.tensor(off, dtype=torch.int32).cuda()
    cache = api.KVCache(kc, vc, table.cuda(), length)
    qo = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    api.kv_append(cache, k, v, seq_off=offs, q=q, q_out=qo, q_norm=qn, k_norm=kn, freq=freq)
    got = f(qo)
    assert (got[n:] == 7).all()
    close(got[:n], ref[0][:n], act)
    close(f(kc), ref[1], act)
    assert np.array_equal(f(vc), ref[2])
    untouched = torch.from_numpy((ref[2] == f(before[1])).all(-1)).cuda()
    assert torch.equal(kc[untouched], before[0][untouched])
    # without queries; one token for each sequence without offsets
    kc2, vc2 = before[0].clone(), before[1].clone()
    api.kv_append(api.KVCache(kc2, vc2, cache.table, length), k, v, seq_off=offs, k_norm=kn, freq=freq)
    assert torch.equal(kc2, kc) and torch.equal(vc2, vc)
    if all(m == 1 for m in new):
        kc2, vc2, qo2 = before[0].clone(), before[1].clone(), torch.empty_like(qo[:n])
        api.kv_append(api.KVCache(kc2, vc2, cache.table, length), k[:n], v[:n], q=q[:n], q_out=qo2, q_norm=qn, k_norm=kn,
                      freq=freq)
        assert torch.equal(kc2, kc) and torch.equal(vc2, vc) and torch.equal(qo2, qo[:n])


def test_append_leaves_out_what_has_no_place():
    import torch
    from int4_routed_expert_router_amd import api
    kc = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.tensor([[0, 1, 9], [2, -1, 3]], dtype=torch.int32).cuda()
    length = torch.tensor([2, 40], dtype=torch.int32).cuda()
    off = torch.tensor([0, 4, 14], dtype=torch.int32).cuda()
    x = torch.full((15, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    qo = torch.full_like(x, 7.0)
    api.kv_append(api.KVCache(kc, vc, table, length), x, x, seq_off=off, q=x, q_out=qo)
    assert (qo[:2] == 7).all() and (qo[2:14] == 3).all() and (qo[14] == 7).all()
    for t in (kc, vc):
        want = torch.zeros_like(t)
        want[0, :, :2] = 3          # positions 0 and 1 of sequence 0
        want[3, :, :8] = 3          # positions 32 .. 39 of sequence 1; 30 and 31 have no page
        assert torch.equal(t, want)


def test_append_in_place_and_at_far_positions():
    import torch
    from int4_routed_expert_router_amd import api
    from oracle import attention_oracle as ao
    pos = [0, 1, 1000003, (1 << 30) - 1]
    n_pages, d = 4, 128
    kc = torch.zeros(n_pages, 2, 256, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.full((4, 1 << 22), -1, dtype=torch.int32, device="cuda")
    for b, p in enumerate(pos):
        table[b, p // 256] = b
    q, k, v, qn, kn, freq = append_inputs(4, 2, d, 4, d, True, "bf16", 5)
    length = torch.tensor([p + 1 for p in pos], dtype=torch.int32).cuda()
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    ref = np.stack([ao._head(f(q)[i], f(qn), 1e-6, f(freq), p) for i, p in enumerate(pos)])
    q = q.contiguous()
    api.kv_append(api.KVCache(kc, vc, table, length), k, v, q=q, q_out=q, q_norm=qn, k_norm=kn, freq=freq)
    close(f(q), ref, "bf16")
    close(f(torch.stack([kc[b, :, p % 256] for b, p in enumerate(pos)])),
          np.stack([ao._head(f(k)[i], f(kn), 1e-6, f(freq), p) for i, p in enumerate(pos)]), "bf16")


def test_append_of_rows_whose_squares_overflow():
    import torch
    from int4_routed_expert_router_amd import api
    kc = torch.ones(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.ones_like(kc)
    x = torch.full((1, 1, 64), 2.0 ** 100, dtype=torch.bfloat16, device="cuda")
    w, freq = torch.ones(64, device="cuda"), torch.ones(8, dtype=torch.float64, device="cuda")
    api.kv_append(api.KVCache(kc, vc, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                              torch.ones(1, dtype=torch.int32, device="cuda")), x, x, k_norm=w, freq=freq)
    assert not kc[0, 0, 0].any() and (vc[0, 0, 0] == 2.0 ** 100).all() and (kc[0, 0, 1:] == 1).all()


# ------------------------------------------------------------------ refusals of the binding
def test_refusals():
    import torch
    from int4_routed_expert_router_amd import MoeError, api
    c = case([2, 1], [20, 3], 4, 2, 64, 16, "bf16", gate=True)
    cache, o = c.cache(), torch.empty(c.q.shape, dtype=c.q.dtype, device="cuda")
    q, off = c.q, c.off

    def refused(fn, match, kind=ValueError):
        with pytest.raises(kind, match=match):
            fn()

    refused(lambda: api.KVCache(c.k, c.v.half(), c.table, c.length), "dtype")
    refused(lambda: api.KVCache(c.k.float(), c.v.float(), c.table, c.length), "float16 or bfloat16")
    refused(lambda: api.KVCache(c.k, c.v[:2], c.table, c.length), "shape")
    refused(lambda: api.KVCache(c.k.transpose(1, 2), c.v.transpose(1, 2), c.table, c.length), "contiguous")
    refused(lambda: api.KVCache(c.k, c.v, c.table.long(), c.length), "dtype")
    refused(lambda: api.KVCache(c.k, c.v, c.table, c.length[:1]), "length")
    refused(lambda: api.KVCache(c.k, c.v, c.table, c.length.cpu()), "CUDA")
    refused(lambda: api.attn_prefill(cache, q.half(), o, off, 1.0), "dtype")
    refused(lambda: api.attn_prefill(cache, q[..., :32], o, off, 1.0), "shape")
    refused(lambda: api.attn_prefill(cache, q, o[:2], off, 1.0), "o must be")
    refused(lambda: api.attn_prefill(cache, q, o.transpose(0, 1), off, 1.0), "contiguous")
    refused(lambda: api.attn_prefill(cache, q, o, off[:2], 1.0), "elements")
    refused(lambda: api.attn_prefill(cache, q, o, off, 1.0, gate=c.gate[:2]), "shape")
    refused(lambda: api.attn_prefill(cache, q.transpose(1, 2).contiguous().transpose(1, 2), o, off, 1.0), "next to each other")
    refused(lambda: api.attn_prefill(cache, q, o, off, float("nan")), "scale", MoeError)
    refused(lambda: api.attn_prefill(cache, q, o, off, 1.0, ws=torch.empty(1, dtype=torch.uint8, device="cuda")), "workspace",
            MoeError)
    refused(lambda: api.attn_prefill(cache, torch.zeros(5, 3, 64, dtype=c.q.dtype, device="cuda"),
                                     torch.zeros(5, 3, 64, dtype=c.q.dtype, device="cuda"), off, 1.0), "q_heads", MoeError)
    refused(lambda: api.attn_decode(cache, q, o, 1.0), "one for each")
    odd = torch.zeros(5, 4, 65, dtype=c.q.dtype, device="cuda")
    refused(lambda: api.attn_prefill(cache, odd[..., :64], o, off, 1.0), "stride", MoeError)
    refused(lambda: api.attn_prefill(cache, odd.view(-1)[1 : 1 + 5 * 4 * 64].view(5, 4, 64), o, off, 1.0), "aligned", MoeError)
    k = torch.zeros(3, 2, 64, dtype=c.q.dtype, device="cuda")
    refused(lambda: api.kv_append(cache, k[:, :1], k[:, :1], seq_off=off), "heads")
    refused(lambda: api.kv_append(cache, k, k[:2], seq_off=off), "shape")
    refused(lambda: api.kv_append(cache, k, k), "without seq_off", MoeError)
    refused(lambda: api.kv_append(cache, k, k, seq_off=off, q=q[:2], q_out=o[:2]), "tokens")
    refused(lambda: api.kv_append(cache, k, k, seq_off=off, q=q[:3]), "q_out must be")
    refused(lambda: api.kv_append(cache, k, k, seq_off=off, q_out=o[:3]), "needs q")
    refused(lambda: api.kv_append(cache, k, k, seq_off=off, k_norm=torch.ones(32, device="cuda")), "elements")
    refused(lambda: api.kv_append(cache, k, k, seq_off=off, freq=torch.ones(4, device="cuda")), "dtype")
    refused(lambda: api.kv_append(cache, k, k, seq_off=off, freq=torch.ones(4, dtype=torch.float64, device="cuda")),
            "rot_dim", MoeError)
    torch.cuda.synchronize()
