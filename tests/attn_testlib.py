"""Inputs of the paged attention tests on the GPU and their comparison with the oracle."""
import numpy as np
import torch

from int4_routed_expert_router_amd import api
from oracle import attention_oracle as ao

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}       # half a step, relative
TINY = {"bf16": 0.0, "f16": 2.0 ** -25}             # half a step of the smallest values


class Case:
    """Caches, tables and rows of sequences with the given new tokens and total
    lengths.  Whatever no token may see is NaN: pages of no sequence, slots
    behind a sequence's length."""

    def __init__(self, new, total, hq, hk, d, page, act, gate=False, seed=0, spread=1.5, width=None, extra=3, fill=True):
        g = torch.Generator().manual_seed(seed)
        self.new, self.total, self.act, self.page = new, total, act, page
        pages = [-(-t // page) for t in total]
        width = width or max(pages + [0]) + 1
        n_pages = sum(pages) + extra
        order = torch.randperm(n_pages, generator=g).int()
        table = torch.full((len(new), width), -1, dtype=torch.int32)
        k = torch.full((n_pages, hk, page, d), float("nan"))
        v = k.clone()
        at = 0
        for b, n in enumerate(total):
            table[b, : pages[b]] = order[at : at + pages[b]]
            at += pages[b]
            for i in range(pages[b] if fill else 0):
                m = min(page, n - i * page)
                k[table[b, i], :, :m] = torch.randn(hk, m, d, generator=g)
                v[table[b, i], :, :m] = torch.randn(hk, m, d, generator=g) + 0.5
        dt = DT[act]
        self.k, self.v, self.table = k.to(dt).cuda(), v.to(dt).cuda(), table.cuda()
        self.length = torch.tensor(total, dtype=torch.int32).cuda()
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        self.n = sum(new)
        rows = torch.randn(self.n + 2, hq, 2, d, generator=g)   # two rows that no sequence owns
        rows[:, :, 0] *= spread
        rows = rows.to(dt).cuda()
        self.q, self.gate = rows[:, :, 0], rows[:, :, 1] if gate else None
        self.scale = d ** -0.5
        self.weight_step = STEP[act]   # weights may be held in act_dtype

    def cache(self):
        return api.KVCache(self.k, self.v, self.table, self.length)

    def run(self, decode=False, ws=None, stream=None):
        """o with 7 in every row before the call."""
        c = self.cache()
        if decode:
            n = len(self.new)
            o = torch.full(self.q[:n].shape, 7.0, dtype=self.q.dtype, device="cuda")
            api.attn_decode(c, self.q[:n], o, self.scale, gate=None if self.gate is None else self.gate[:n], ws=ws,
                            stream=stream)
        else:
            o = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device="cuda")
            api.attn_prefill(c, self.q, o, self.off, self.scale, gate=self.gate, ws=ws, stream=stream)
        return o

    def check(self, o, decode=False):
        f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        n = len(self.new) if decode else self.q.shape[0]
        q, gate = f(self.q)[:n], f(self.gate)
        off = None if decode else self.off.cpu().numpy()
        ref, bound = ao.attend(f(self.k), f(self.v), self.table.cpu().numpy(), self.length.cpu().numpy(), off, q,
                               self.scale, gate=None if gate is None else gate[:n], weight_step=self.weight_step)
        got = f(o)
        none = np.isnan(ref)
        assert np.array_equal(got[none], np.full(none.sum(), 7.0)), "rows that no sequence owns were written"
        tol = bound + STEP[self.act] * (np.abs(ref) + bound) + TINY[self.act]
        bad = ~(np.abs(got - ref) <= tol) & ~none
        worst = np.nanmax(np.where(none, 0, np.abs(got - ref) / np.maximum(tol, 1e-30)), initial=0)
        assert not bad.any(), f"{bad.sum()} of {bad.size} values off, worst {worst:.3g} of the tolerance, at {np.argwhere(bad)[:3].tolist()}"
