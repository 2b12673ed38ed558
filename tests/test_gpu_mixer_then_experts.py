"""GPU run of the operators together, as a linear-attention layer uses them over
a batch of sequences: int4 projections of the hidden rows to q, k, v and the
gates, Gated DeltaNet over the sequences, the output projection, scored expert
choice and the expert FFN.  Each stage is held to the fp64 oracle on the input
that it was really given, and a captured run to the eager one, bit for bit."""
import dataclasses

import numpy as np
import pytest

from oracle import deltanet_oracle as dn
from oracle import linear_oracle as lo
from oracle import moe_oracle as mo
from oracle import select_oracle as so

pytestmark = pytest.mark.gpu

HK, HV, DV, GROUP = 2, 4, 48, 64
Q_SCALE = 128 ** -0.5


class Layer:
    def __init__(self, lens, seed):
        import synth
        import torch
        from int4_routed_expert_router_amd import api
        from moe_testlib import DeviceLayer, desc_for
        self.wl = dataclasses.replace(synth.TINY, n_experts=24, top_k=6)
        self.H, self.T, self.lens = self.wl.hidden, sum(lens), lens
        rng = np.random.default_rng(seed)
        self.raw, self.lin = {}, {}
        for name, k, n in (("q", self.H, HK * 128), ("k", self.H, HK * 128), ("v", self.H, HV * DV),
                           ("gates", self.H, 2 * HV), ("out", HV * DV, self.H)):
            q = rng.integers(0, 16, (n, k))
            s = (rng.uniform(0.2, 1.2, (n, k // GROUP)) / 40).astype(np.float16)
            b = (-7.5 * s * rng.uniform(0.8, 1.2, s.shape)).astype(np.float16)
            self.raw[name] = (q, s, b)
            self.lin[name] = api.Linear(k, n, GROUP, torch.from_numpy(lo.pack_words(q)).cuda(),
                                        torch.from_numpy(s).cuda(), torch.from_numpy(b).cuda(), act_dtype="f16")
        self.dl = DeviceLayer(self.wl, 0, router_scale=20.0)
        self.bias = (0.3 * rng.standard_normal(24)).astype(np.float32)
        self.dl.router_bias = torch.from_numpy(self.bias).cuda()
        self.desc, self.sel = desc_for(self.wl), api.SelectDesc(24, 6, "sigmoid", 4, 2, 2, True, 2.5)
        e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        T, h = self.T, torch.float16
        self.x = torch.from_numpy(rng.standard_normal((T, self.H)).astype(np.float32)).cuda().to(h)
        self.state0 = torch.from_numpy(0.3 * rng.standard_normal((len(lens), HV, DV, 128))).float().cuda()
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        self.ws = api.gdn_prefill_workspace(len(lens), T, HK, HV, DV, "f16")
        self.b = dict(q=e(T, HK, 128, t=h), k=e(T, HK, 128, t=h), v=e(T, HV, DV, t=h), gates=e(T, 2 * HV),
                      g=e(T, HV), beta=e(T, HV), state=e(len(lens), HV, DV, 128), o=e(T, HV, DV),
                      o16=e(T, HV * DV, t=h), mixed=e(T, self.H), x2=e(T, self.H, t=h),
                      idx=e(T, 6, t=torch.int32), w=e(T, 6), gamma=e(T), logits=e(T, 25), y=e(T, self.H))

    def run(self):
        import torch
        from int4_routed_expert_router_amd import api
        b = self.b
        for name in ("q", "k", "v", "gates"):
            api.linear(self.lin[name], self.x, b[name])
        b["g"].copy_(-torch.nn.functional.softplus(b["gates"][:, :HV]))
        b["beta"].copy_(torch.sigmoid(b["gates"][:, HV:]))
        b["state"].copy_(self.state0)
        api.gdn_prefill(b["q"], b["k"], b["v"], b["g"], b["beta"], b["state"], b["o"], self.off, Q_SCALE, "f16",
                        ws=self.ws)
        b["o16"].copy_(b["o"].view(self.T, -1))
        api.linear(self.lin["out"], b["o16"], b["mixed"])
        b["x2"].copy_(b["mixed"] + self.x.float())
        api.route_scored(self.desc, self.sel, self.dl.api_layer(), b["x2"], b["idx"], b["w"], b["gamma"], b["logits"])
        api.expert_ffn(self.desc, self.dl.api_layer(), b["x2"], b["idx"], b["w"], b["gamma"], b["y"])

    def host(self):
        import torch
        torch.cuda.synchronize()
        return {k: v.cpu().numpy().copy() for k, v in self.b.items()}


@pytest.mark.parametrize("lens", [[1, 1, 1], [30, 0, 70, 3]], ids=["decode", "prompts"])
def test_every_stage_against_its_oracle(lens):
    m = Layer(lens, 5)
    m.run()
    r = m.host()

    def product(name, x, got):   # fp32 bound of the sums, then one rounding to the output's type
        x = x.astype(np.float64)
        ref, tol = lo.linear(x, *m.raw[name], GROUP), lo.error_bound(x, *m.raw[name], GROUP)
        half = 2.0 ** -11 if got.dtype == np.float16 else 2.0 ** -24
        err = np.abs(got.reshape(ref.shape).astype(np.float64) - ref)
        assert (err <= tol + half * (np.abs(ref) + tol) + 2.0 ** -25).all(), name

    x = m.x.cpu().numpy()
    for name in ("q", "k", "v", "gates"):
        product(name, x, r[name])
    f = {k: r[k].astype(np.float64) for k in ("q", "k", "v", "g", "beta")}
    S, o = dn.gdn_sequences(m.state0.cpu().numpy().astype(np.float64), f["q"], f["k"], f["v"], f["g"], f["beta"],
                            Q_SCALE, lens)
    # a few dozen fp32 roundings per output, for each of up to 70 tokens that a
    # state remembers: 8 x 2^-24 sqrt(70) of the whole output's 2-norm
    for got, want in ((r["o"], o), (r["state"], S)):
        assert np.linalg.norm(got - want) <= 8 * 2.0 ** -24 * 70 ** 0.5 * np.linalg.norm(want)
    product("out", r["o16"], r["mixed"])
    x2 = r["x2"].astype(np.float64)
    z64, _ = mo.router_logits(x2, m.dl.router_f64(), None)
    assert np.abs(r["logits"][:, :24] - z64).max() <= 1e-5 * np.abs(z64).max()
    ref_i, ref_w = so.select(r["logits"][:, :24], 6, "sigmoid", m.bias, n_group=4, top_groups=2, group_top=2, scale=2.5)
    assert np.array_equal(r["idx"], ref_i)
    assert (np.abs(r["w"] - ref_w) <= 1.01 * 2.0 ** -24 * ref_w).all()
    gate = 1 / (1 + np.exp(-r["logits"][:, 24].astype(np.float64)))
    ex = {e: m.dl.oracle_expert(e) for e in sorted(set(ref_i.ravel().tolist()))}
    sh, ref_y = m.dl.oracle_shared(), np.zeros((m.T, m.H))
    for t in range(m.T):
        ref_y[t] = gate[t] * mo.expert_ffn(x2[t], sh.wg, sh.wu, sh.wd)
        for e, we in zip(ref_i[t], ref_w[t]):
            ref_y[t] += we * mo.expert_ffn(x2[t], ex[e].wg, ex[e].wu, ex[e].wd)
    from moe_testlib import assert_close
    assert_close(r["y"], ref_y, "y")


@pytest.mark.parametrize("lens", [[5, 2], [30, 0, 70, 3]], ids=["drafts", "prompts"])
def test_captured_run_equals_the_eager_one(lens):
    import torch
    m = Layer(lens, 6)
    first, second = m.x.clone(), (m.x.float() * 0.5 + 0.25).to(m.x.dtype)
    want = []
    for x in (first, second):
        m.x.copy_(x)
        m.run()
        want.append(m.host())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.run()
    for i in (0, 1, 1, 0):
        m.x.copy_(first if i == 0 else second)
        for t in m.b.values():
            t.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        got = m.host()
        for k, v in want[i].items():
            assert np.array_equal(got[k], v), (i, k)
        m.run()   # eager work between the replays
        torch.cuda.synchronize()
