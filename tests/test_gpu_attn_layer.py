"""GPU run of the operators of a gated attention layer together: one int4
projection of the hidden rows to queries, gates, keys and values, the cache
append with norms and rotary positions on slices of its output, attention over
the pages, the output projection, scored expert choice and the experts.  A
conversation is a prompt, more turns and single tokens.  Each stage is held to
its fp64 oracle on the input that it was really given, and a captured step to
the eager one, bit for bit."""
import dataclasses

import numpy as np
import pytest

from oracle import attention_oracle as ao
from oracle import linear_oracle as lo
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE, ROT, GROUP, EPS = 6, 2, 64, 16, 32, 64, 1e-6
STEP = 2.0 ** -11   # half a step of fp16, relative


class Layer:
    def __init__(self, batch, seed, width=20):
        import synth
        import torch
        from int4_routed_expert_router_amd import api
        from moe_testlib import DeviceLayer, desc_for
        self.wl = dataclasses.replace(synth.TINY, n_experts=24, top_k=6)
        self.H, self.B = self.wl.hidden, batch
        rng = np.random.default_rng(seed)
        self.raw, self.lin = {}, {}
        for name, k, n in (("in", self.H, (2 * HQ + 2 * HK) * D), ("out", HQ * D, self.H)):
            q = rng.integers(0, 16, (n, k))
            s = (rng.uniform(0.2, 1.2, (n, k // GROUP)) / 40).astype(np.float16)
            b = (-7.5 * s * rng.uniform(0.8, 1.2, s.shape)).astype(np.float16)
            self.raw[name] = (q, s, b)
            self.lin[name] = api.Linear(k, n, GROUP, torch.from_numpy(lo.pack_words(q)).cuda(),
                                        torch.from_numpy(s).cuda(), torch.from_numpy(b).cuda(), act_dtype="f16")
        self.dl = DeviceLayer(self.wl, 0, router_scale=20.0)
        self.desc, self.sel = desc_for(self.wl), api.SelectDesc(24, 6, "sigmoid", 4, 2, 2, True, 2.5)
        self.qn, self.kn = (torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).float().cuda() for _ in range(2))
        self.freq = 1e4 ** (-2 * torch.arange(ROT // 2, dtype=torch.float64, device="cuda") / ROT)
        pages = batch * width
        k, v = (torch.full((pages, HK, PAGE, D), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
        table = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda().view(batch, width)
        self.cache = api.KVCache(k, v, table, torch.zeros(batch, dtype=torch.int32, device="cuda"))
        self.ws = api.attn_workspace(self.cache, HQ, 400)
        self.rng = rng

    def buffers(self, new):
        import torch
        T = sum(new)
        e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        h = torch.float16
        x = torch.from_numpy(self.rng.standard_normal((T, self.H)).astype(np.float32)).cuda().to(h)
        off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        return dict(x=x, off=off, rows=e(T, (2 * HQ + 2 * HK) * D, t=h), q=e(T, HQ, D, t=h), o=e(T, HQ, D, t=h),
                    mixed=e(T, self.H), x2=e(T, self.H, t=h), idx=e(T, 6, t=torch.int32), w=e(T, 6), gamma=e(T),
                    logits=e(T, 25), y=e(T, self.H))

    def run(self, b, decode):
        from int4_routed_expert_router_amd import api
        T = b["x"].shape[0]
        api.linear(self.lin["in"], b["x"], b["rows"])
        qg = b["rows"][:, : 2 * HQ * D].view(T, HQ, 2, D)
        k, v = b["rows"][:, 2 * HQ * D :].view(T, 2, HK, D).unbind(1)
        api.kv_append(self.cache, k, v, seq_off=None if decode else b["off"], q=qg[:, :, 0], q_out=b["q"],
                      q_norm=self.qn, k_norm=self.kn, eps=EPS, freq=self.freq)
        if decode:
            api.attn_decode(self.cache, b["q"], b["o"], D ** -0.5, gate=qg[:, :, 1], ws=self.ws)
        else:
            api.attn_prefill(self.cache, b["q"], b["o"], b["off"], D ** -0.5, gate=qg[:, :, 1], ws=self.ws)
        api.linear(self.lin["out"], b["o"].view(T, -1), b["mixed"])
        b["x2"].copy_(b["mixed"] + b["x"].float())
        api.route_scored(self.desc, self.sel, self.dl.api_layer(), b["x2"], b["idx"], b["w"], b["gamma"], b["logits"])
        api.expert_ffn(self.desc, self.dl.api_layer(), b["x2"], b["idx"], b["w"], b["gamma"], b["y"])

    def product(self, name, x, got):
        x = x.astype(np.float64)
        ref, tol = lo.linear(x, *self.raw[name], GROUP), lo.error_bound(x, *self.raw[name], GROUP)
        half = STEP if got.dtype == np.float16 else 2.0 ** -24
        err = np.abs(got.reshape(ref.shape).astype(np.float64) - ref)
        assert (err <= tol + half * (np.abs(ref) + tol) + 2.0 ** -25).all(), name


def step(m, new, decode=False):
    """One call of the layer, every stage checked."""
    import torch
    from moe_testlib import assert_close
    from test_gpu_attn import close
    b = m.buffers(new)
    before = [t.double().cpu().numpy() for t in (m.cache.k, m.cache.v)]
    m.cache.length.add_(torch.tensor(new, dtype=torch.int32, device="cuda"))
    m.run(b, decode)
    torch.cuda.synchronize()
    r = {k: v.cpu().numpy() for k, v in b.items()}
    m.product("in", r["x"], r["rows"])
    T = len(r["x"])
    f = r["rows"].astype(np.float64)
    qg, kv = f[:, : 2 * HQ * D].reshape(T, HQ, 2, D), f[:, 2 * HQ * D :].reshape(T, 2, HK, D)
    table, length, off = m.cache.table.cpu().numpy(), m.cache.length.cpu().numpy(), r["off"]
    q, kc, vc = ao.append(*before, table, length, off, kv[:, 0], kv[:, 1], qg[:, :, 0], m.qn.double().cpu().numpy(),
                          m.kn.double().cpu().numpy(), EPS, m.freq.cpu().numpy())
    close(r["q"].astype(np.float64), q, "f16")
    after = [t.double().cpu().numpy() for t in (m.cache.k, m.cache.v)]
    live = ~np.isnan(kc)
    assert np.array_equal(np.isnan(after[0]), ~live) and np.array_equal(after[1], vc, equal_nan=True)
    close(np.where(live, after[0], 0), np.where(live, kc, 0), "f16")
    o, bound = ao.attend(*after, table, length, off, r["q"].astype(np.float64), D ** -0.5, gate=qg[:, :, 1],
                         weight_step=STEP)
    assert (np.abs(r["o"] - o) <= bound + STEP * (np.abs(o) + bound) + 2.0 ** -25).all()
    m.product("out", r["o"].reshape(T, -1), r["mixed"])
    x2 = r["x2"].astype(np.float64)
    z64, _ = mo.router_logits(x2, m.dl.router_f64(), None)
    assert np.abs(r["logits"][:, :24] - z64).max() <= 1e-5 * np.abs(z64).max()
    gate = 1 / (1 + np.exp(-r["logits"][:, 24].astype(np.float64)))
    sh, ref_y = m.dl.oracle_shared(), np.zeros((T, m.H))
    ex = {e: m.dl.oracle_expert(e) for e in sorted(set(r["idx"].ravel().tolist()))}
    for t in range(T):
        ref_y[t] = gate[t] * mo.expert_ffn(x2[t], sh.wg, sh.wu, sh.wd)
        for e, we in zip(r["idx"][t], r["w"][t].astype(np.float64)):
            ref_y[t] += we * mo.expert_ffn(x2[t], ex[e].wg, ex[e].wu, ex[e].wd)
    assert_close(r["y"], ref_y, "y")


def test_a_conversation_stage_by_stage():
    m = Layer(3, 1)
    step(m, [40, 3, 0])                  # prompts
    step(m, [1, 20, 33])                 # more turns over what is cached
    step(m, [1, 1, 1], decode=True)      # single tokens
    step(m, [5, 5, 5])                   # drafted tokens
    step(m, [1, 1, 1], decode=True)
    assert m.cache.length.tolist() == [48, 30, 40]


def test_pieces_of_a_prompt_and_single_tokens_agree_with_the_whole():
    # the same rows through the cache in one call, in pieces, and token by token: the keys and values are the same bits,
    # the outputs the same up to the order of sums
    import torch
    from int4_routed_expert_router_amd import api
    n, outs, caches = 70, [], []
    for pieces in ([70], [1, 16, 33, 20], [1] * 70):
        m = Layer(1, 2)
        rows = torch.randn(n, (HQ + 2 * HK), D, generator=torch.Generator().manual_seed(3)).half().cuda()
        out = torch.empty(n, HQ, D, dtype=torch.float16, device="cuda")
        at = 0
        for p in pieces:
            m.cache.length.add_(p)
            x = rows[at : at + p]
            q = torch.empty(p, HQ, D, dtype=torch.float16, device="cuda")
            off = torch.tensor([0, p], dtype=torch.int32, device="cuda")
            api.kv_append(m.cache, x[:, HQ : HQ + HK], x[:, HQ + HK :], seq_off=off, q=x[:, :HQ], q_out=q, q_norm=m.qn,
                          k_norm=m.kn, freq=m.freq)
            if len(pieces) == n:
                api.attn_decode(m.cache, q, out[at : at + 1], D ** -0.5)
            else:
                api.attn_prefill(m.cache, q, out[at : at + p], off, D ** -0.5)
            at += p
        outs.append(out.double())
        caches.append((m.cache.k.clone(), m.cache.v.clone()))
    for k, v in caches[1:]:
        assert torch.equal(k.isnan(), caches[0][0].isnan()) and torch.equal(k.nan_to_num(), caches[0][0].nan_to_num())
        assert torch.equal(v.nan_to_num(), caches[0][1].nan_to_num())
    # each is within half a step of the output and half a step of each weight of the true value
    big = caches[0][1].nan_to_num().abs().max().double()
    for o in outs[1:]:
        assert ((o - outs[0]).abs() <= 2 * STEP * (outs[0].abs() + big) + 2.0 ** -14).all()


def test_a_captured_step_of_growing_sequences():
    # one graph for every step: lengths grow on the device between replays
    import torch
    m = Layer(4, 7)
    first = m.buffers([30, 1, 0, 17])
    m.cache.length.copy_(torch.tensor([30, 1, 0, 17], dtype=torch.int32))
    m.run(first, False)
    b = m.buffers([1, 1, 1, 1])
    xs = [torch.randn(4, m.H, device="cuda").half() for _ in range(4)]
    start = [t.clone() for t in (m.cache.k, m.cache.v, m.cache.length)]

    def restore():
        for t, s in zip((m.cache.k, m.cache.v, m.cache.length), start):
            t.copy_(s)

    def steps(call):
        outs = []
        for x in xs:
            m.cache.length.add_(1)
            b["x"].copy_(x)
            for k, t in b.items():
                if k not in ("x", "off"):
                    t.fill_(7)
            call()
            torch.cuda.synchronize()
            outs.append({k: t.clone() for k, t in b.items()})
        return outs + [{"k": m.cache.k.nan_to_num(), "v": m.cache.v.nan_to_num()}]

    want = steps(lambda: m.run(b, True))
    restore()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.run(b, True)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.run(b, True)
    for _ in range(2):
        restore()
        got = steps(g.replay)
        for i, (x, y) in enumerate(zip(got, want)):
            for k in y:
                assert torch.equal(x[k], y[k]), (i, k)
        restore()
        m.run(first, False)   # eager work between the replays
        torch.cuda.synchronize()
