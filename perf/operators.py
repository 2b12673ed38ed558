"""Three operators around the int4 routed-expert layer, in plain torch and as the framework's own calls.

  linear  y = x W^T with W[r,c] = s[r,c/G] q[r,c] + b[r,c/G], q in 0..15: the dense projections beside the experts
          (queries, keys, values and outputs of the token mixers, the vocabulary projection), one token to a prompt's worth
  select  top-K of E experts from router logits: softmax or sigmoid scores, a balance bias that enters the choice but
          not the weights, group-limited choice, renormalised and scaled weights
  gdn     the gated delta rule over whole prompts of several sequences, packed one after the other, with the state
          carried in and out (the decode step's rule, applied token after token)
"""
import math
import random

import torch

own = False


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a mixer's input projection: latency
        dict(name="linear_decode", op="linear", tokens=1, inp=2048, out=8192, group=64, act="bf16", res="bf16"),
        # one token through a vocabulary projection of an odd size, logits in 32 bits
        dict(name="linear_vocab", op="linear", tokens=1, inp=2048, out=100003, group=64, act="bf16", res="f32"),
        # a few sequences, narrow odd output (gates of the heads), fp16
        dict(name="linear_gates", op="linear", tokens=5, inp=2048, out=65, group=32, act="f16", res="f32"),
        # a decode batch through an output projection
        dict(name="linear_batch", op="linear", tokens=64, inp=4096, out=2048, group=64, act="bf16", res="bf16"),
        # part of a prompt, odd token count
        dict(name="linear_prompt", op="linear", tokens=499, inp=2048, out=8192, group=128, act="f16", res="f16"),
        # one decode token, 10 of 512, the softmax form
        dict(name="select_decode", op="select", tokens=1, experts=512, k=10, score="softmax", groups=1, top_groups=1,
             group_top=1, renorm=True, bias=False, scale=1.0),
        # a decode batch, sigmoid scores, balance bias, 4 of 8 groups
        dict(name="select_batch", op="select", tokens=64, experts=256, k=8, score="sigmoid", groups=8, top_groups=4,
             group_top=2, renorm=True, bias=True, scale=2.5),
        # a prompt, the same routing
        dict(name="select_prompt", op="select", tokens=8191, experts=256, k=8, score="sigmoid", groups=8, top_groups=4,
             group_top=2, renorm=True, bias=True, scale=2.5),
        # one short continuation (five drafted tokens), 16 key and 32 value heads
        dict(name="gdn_draft", op="gdn", seqs=1, tokens=5, k_heads=16, v_heads=32, dv=128, act="bf16"),
        # a batch of prompts of very different lengths
        dict(name="gdn_prompts", op="gdn", seqs=12, tokens=6001, k_heads=16, v_heads=32, dv=128, act="bf16"),
        # one long prompt
        dict(name="gdn_long", op="gdn", seqs=1, tokens=8192, k_heads=16, v_heads=32, dv=128, act="bf16"),
        # a small layer: fp16, few heads, a narrow value head
        dict(name="gdn_small", op="gdn", seqs=3, tokens=700, k_heads=2, v_heads=6, dv=48, act="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "select", "gdn"))
    if op == "linear":
        group = rng.choice((32, 64, 128))
        unit = max(group, 64)
        inp = unit * max(1, _log(rng, 64, 8192) // unit)
        out = _log(rng, 1, 65536)
        tokens = _log(rng, 1, 512)
        tokens = max(1, min(tokens, 499 * 2048 * 8192 // (inp * out)))
        return dict(op=op, tokens=tokens, inp=inp, out=out, group=group, act=rng.choice(("bf16", "f16")),
                    res=rng.choice(("bf16", "f16", "f32")))
    if op == "select":
        groups = rng.choice((1, 1, 2, 4, 5, 8, 16))
        per = _log(rng, 2, 1024 // groups)
        top_groups = rng.randint(1, groups)
        k = min(rng.randint(1, 32), top_groups * per)
        tokens = min(_log(rng, 1, 16384), 8191 * 256 // (groups * per))
        return dict(op=op, tokens=tokens, experts=groups * per, k=k, score=rng.choice(("softmax", "sigmoid")),
                    groups=groups, top_groups=top_groups, group_top=rng.choice((1, 2)), renorm=rng.random() < 0.7,
                    bias=rng.random() < 0.6, scale=rng.choice((1.0, 2.5, 16.0)))
    k_heads = rng.choice((1, 2, 3, 4, 8, 16))
    v_heads = k_heads * rng.choice((1, 2, 3, 4))
    dv = rng.choice((16, 48, 64, 128, 128, 256))
    tokens = max(1, min(_log(rng, 1, 12000), 8192 * 32 * 128 // (v_heads * dv)))
    return dict(op=op, seqs=min(_log(rng, 1, 32), tokens), tokens=tokens, k_heads=k_heads, v_heads=v_heads, dv=dv,
                act=rng.choice(("bf16", "f16")))


_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _lengths(case):
    """Sequence lengths of a packed batch: uneven, adding up to the case's tokens; a batch of many holds an empty one."""
    n, total = case["seqs"], case["tokens"]
    r = random.Random(n * 1000003 + total)
    cuts = sorted(int(total * r.random() ** 1.5) for _ in range(n - 1))
    if n > 2:
        cuts[1] = cuts[0]
    ends = [0] + cuts + [total]
    return [b - a for a, b in zip(ends, ends[1:])]


# --------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    if case["op"] == "linear":
        n, k, g = case["out"], case["inp"], case["group"]
        words = torch.randint(-2 ** 31, 2 ** 31, (n, k // 8), generator=gen, device="cuda").to(torch.int32)
        scale = ((0.2 + rand(n, k // g)) * (1.5 / (4.6 * math.sqrt(k)))).half()
        bias = (-7.5 * scale.float() * (0.9 + 0.2 * rand(n, k // g))).half()
        return dict(words=words, scale=scale, bias=bias, x=randn(case["tokens"], k).to(_DT[case["act"]]))
    if case["op"] == "select":
        t, e = case["tokens"], case["experts"]
        logits = 1.2 * randn(t, e) + randn(e)
        bias = 0.2 * randn(e) if case["bias"] else None
        if e > 4:   # an expert out of service for some tokens
            logits[:: 3, 3] = float("-inf")
        return dict(logits=logits.contiguous(), bias=bias)
    n, hk, hv, dv = case["tokens"], case["k_heads"], case["v_heads"], case["dv"]
    silu = torch.nn.functional.silu
    dt = _DT[case["act"]]
    lens = _lengths(case)
    off = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    rate = torch.exp(math.log(0.002) + rand(hv) * (math.log(8.0) - math.log(0.002)))
    return dict(q=silu(randn(n, hk, 128)).to(dt), k=silu(randn(n, hk, 128)).to(dt), v=silu(randn(n, hv, dv)).to(dt),
                g=-(rate * torch.nn.functional.softplus(randn(n, hv))), beta=torch.sigmoid(1.5 * randn(n, hv)),
                state=0.3 * randn(len(lens), hv, dv, 128), off=off, lens=lens, q_scale=1.0 / math.sqrt(128))


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if case["op"] == "linear":
        s["y"] = torch.empty(case["tokens"], case["out"], dtype=_DT[case["res"]], device="cuda")
    elif case["op"] == "select":
        s["idx"] = torch.empty(case["tokens"], case["k"], dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(case["tokens"], case["k"], device="cuda")
    else:
        s["o"] = torch.empty(case["tokens"], case["v_heads"], case["dv"], device="cuda")
    if own:
        from int4_routed_expert_router_amd import api
        s["api"] = api
        if case["op"] == "linear":   # the weights are laid out once, when a program loads them
            s["linear"] = api.Linear(case["inp"], case["out"], case["group"], s["words"], s["scale"], s["bias"],
                                     act_dtype=case["act"])
        elif case["op"] == "select":
            s["desc"] = api.SelectDesc(case["experts"], case["k"], score=case["score"], n_group=case["groups"],
                                       top_groups=case["top_groups"], group_top=case["group_top"],
                                       renorm=case["renorm"], scale=case["scale"])
        else:
            s["ws"] = api.gdn_prefill_workspace(case["seqs"], case["tokens"], case["k_heads"], case["v_heads"],
                                                case["dv"], act_dtype=case["act"])
    return s


# --------------------------------------------------------------------------- plain forms
def _linear_plain(s):
    c = s["case"]
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device="cuda")
    q = (s["words"].unsqueeze(-1) >> shifts) & 15                       # value 8 i + j in bits 4 j of word i
    q = q.view(c["out"], c["inp"] // c["group"], c["group"]).float()
    w = q * s["scale"].float().unsqueeze(-1) + s["bias"].float().unsqueeze(-1)
    s["y"].copy_(s["x"].float() @ w.view(c["out"], c["inp"]).t())
    return s["y"]


def _select_plain(s):
    # in 64 bits: two experts whose keys lie next to each other have to come in their true order
    c, ninf = s["case"], float("-inf")
    z = torch.nan_to_num(s["logits"].double(), nan=ninf, posinf=float("inf"), neginf=ninf)
    off = z == ninf
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        top = z.amax(-1, keepdim=True)
        ex = torch.where(z == top, torch.ones_like(z), torch.exp(z - top))
        score = ex / ex.sum(-1, keepdim=True)
    score = torch.where(off, torch.zeros_like(score), score)
    key = score if s["bias"] is None else score + s["bias"].double()
    key = torch.where(off, torch.full_like(key, ninf), key)
    t, per = key.shape[0], c["experts"] // c["groups"]
    if c["top_groups"] < c["groups"]:
        of_group = key.view(t, c["groups"], per)
        best = torch.sort(of_group, dim=-1, descending=True)[0][..., : min(c["group_top"], per)]
        rank = torch.where(best == ninf, torch.zeros_like(best), best).sum(-1)
        rank = torch.where(best[..., 0] == ninf, torch.full_like(rank, ninf), rank)
        keep = torch.sort(rank, dim=-1, descending=True, stable=True)[1][:, : c["top_groups"]]
        mask = torch.zeros(t, c["groups"], dtype=torch.bool, device=key.device).scatter_(1, keep, True)
        key = torch.where(mask.unsqueeze(-1), of_group, torch.full_like(of_group, ninf)).view(t, -1)
    top, idx = (v[:, : c["k"]] for v in torch.sort(key, dim=-1, descending=True, stable=True))
    live = top != ninf
    w = torch.where(live, score.gather(1, idx), torch.zeros_like(top))
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    s["idx"].copy_(torch.where(live, idx, torch.full_like(idx, -1)))
    s["w"].copy_(w * c["scale"])
    return s["idx"], s["w"]


def _gdn_plain(s):
    # chunks of C tokens: with G the running sum of g in the chunk and S the state before it,
    #   (I + A) D = beta V - beta e^G K S^T,  A_ij = beta_i e^(G_i - G_j) k_i.k_j (j < i)
    #   O = e^G Q S^T + P D,  P_ij = e^(G_i - G_j) q_i.k_j (j <= i),  S <- e^G_C S + D^T (e^(G_C - G) K)
    c, C = s["case"], min(64, max(s["lens"]))
    b, n, rep = len(s["lens"]), c["tokens"], c["v_heads"] // c["k_heads"]
    longest = -(-max(s["lens"]) // C) * C
    pos = torch.arange(longest, device="cuda")
    start, end = s["off"][:-1].long().unsqueeze(1), s["off"][1:].long().unsqueeze(1)
    at = torch.where(start + pos < end, start + pos, torch.full_like(pos, n))   # row n: a token that does nothing

    def chunks(x):   # [N, H, ...] -> [chunks, B, H, C, ...]
        x = torch.cat([x, torch.zeros_like(x[:1])])[at]
        x = x.view(b, -1, C, *x.shape[2:]).transpose(0, 1)
        return x.transpose(2, 3).contiguous()

    def unit(x):
        x = x.float()
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)

    q = chunks(unit(s["q"]) * s["q_scale"]).repeat_interleave(rep, 2)
    k = chunks(unit(s["k"])).repeat_interleave(rep, 2)
    v, beta = chunks(s["v"].float()), chunks(s["beta"]).unsqueeze(-1)
    G = chunks(s["g"]).double().cumsum(-1)
    ratio = torch.tril(torch.exp((G.unsqueeze(-1) - G.unsqueeze(-2)).clamp(max=0)).float())
    kt = k.transpose(-1, -2).contiguous()
    A = torch.tril(beta * (k @ kt) * ratio, -1)
    P = (q @ kt) * ratio
    grow, left = torch.exp(G).float().unsqueeze(-1), torch.exp(G[..., -1:] - G).float().unsqueeze(-1)
    inv = torch.eye(C, device="cuda").expand_as(A).contiguous()
    for i in range(1, C):   # rows of (I + A)^-1, from the top
        inv[..., i, :i] = -(A[..., i : i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    S, out = s["state"], []
    for i in range(q.shape[0]):
        st = S.transpose(-1, -2).contiguous()
        d = inv[i] @ (beta[i] * (v[i] - grow[i] * (k[i] @ st)))
        out.append(grow[i] * (q[i] @ st) + P[i] @ d)
        S = grow[i][..., -1:, :] * S + d.transpose(-1, -2).contiguous() @ (left[i] * k[i])
    out = torch.stack(out).permute(1, 0, 3, 2, 4).reshape(b, longest, c["v_heads"], c["dv"])
    s["state"].copy_(S)
    real = at < n
    s["o"][at[real]] = out[real]
    return s["o"], s["state"]


def run(s):
    c = s["case"]
    if not own:
        return {"linear": _linear_plain, "select": _select_plain, "gdn": _gdn_plain}[c["op"]](s)
    if c["op"] == "linear":
        s["api"].linear(s["linear"], s["x"], s["y"])
        return s["y"]
    if c["op"] == "select":
        s["api"].select(s["desc"], s["logits"], s["idx"], s["w"], bias=s["bias"])
        return s["idx"], s["w"]
    s["api"].gdn_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["o"], s["off"], s["q_scale"],
                         act_dtype=c["act"], ws=s["ws"])
    return s["o"], s["state"]


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "linear":
        t, k, n, g = case["tokens"], case["inp"], case["out"], case["group"]
        return {"bytes": n * k / 2 + 4 * n * k / g + 2 * t * k + t * n * (4 if case["res"] == "f32" else 2),
                "flops": 2 * t * k * n}
    if case["op"] == "select":
        t, e = case["tokens"], case["experts"]
        return {"bytes": 4 * t * e + 8 * t * case["k"] + (4 * e if case["bias"] else 0), "flops": 8 * t * e}
    n, hk, hv, dv, b = case["tokens"], case["k_heads"], case["v_heads"], case["dv"], case["seqs"]
    per_head = 4 * n * (2 * 128) + n * 64 * (2 * 2 * 128 + 2 * 2 * dv) / 2 + 3 * 2 * n * 128 * dv
    return {"bytes": n * (4 * hk * 128 + hv * (2 * dv + 8 + 4 * dv)) + 8 * b * hv * dv * 128, "flops": hv * per_head}


# --------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear":
        rows = []
        for r in range(0, case["out"], 16384):   # a block of rows at a time
            words = s["words"][r : r + 16384].long()
            q = torch.stack([(words >> (4 * j)) % 16 for j in range(8)], -1).flatten(1).double()
            spread = lambda m: m[r : r + 16384].double().repeat_interleave(case["group"], 1)  # noqa: E731
            rows.append((spread(s["scale"]) * q + spread(s["bias"])) @ s["x"].double().t().contiguous())
        return torch.cat(rows).t()
    if case["op"] == "select":
        return _select_exact(case, s)
    # token after token: S <- a S + b (v - a S k) k^T, o = S q
    S, rep = s["state"].double(), case["v_heads"] // case["k_heads"]
    unit = lambda x: (x.double() / (x.double().square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(rep, 1)  # noqa: E731
    q, k, v, a, beta = unit(s["q"]) * s["q_scale"], unit(s["k"]), s["v"].double(), s["g"].double().exp(), s["beta"].double()
    o = torch.empty_like(v)
    order = sorted(range(case["seqs"]), key=lambda i: -s["lens"][i])
    first = torch.tensor([sum(s["lens"][:i]) for i in order], device="cuda")
    S = S[order].contiguous()
    for t in range(max(s["lens"])):
        m = sum(n > t for n in s["lens"])   # the longest come first: the first m still have a token
        at = first[:m] + t
        S[:m] *= a[at][..., None, None]
        kk = k[at].unsqueeze(-2)
        S[:m] += (beta[at][..., None] * (v[at] - (S[:m] * kk).sum(-1))).unsqueeze(-1) * kk
        o[at] = (S[:m] * q[at].unsqueeze(-2)).sum(-1)
    back = torch.empty_like(S)
    back[order] = S
    return o, back


def _select_exact(case, s):
    import numpy as np
    z = s["logits"].double().cpu().numpy()
    bias = np.zeros(case["experts"]) if s["bias"] is None else s["bias"].double().cpu().numpy()
    idx, wgt = np.full((case["tokens"], case["k"]), -1, np.int32), np.zeros((case["tokens"], case["k"]))
    per = case["experts"] // case["groups"]
    for t in range(case["tokens"]):
        live = z[t] > -np.inf
        if case["score"] == "sigmoid":
            with np.errstate(over="ignore"):
                score = np.where(live, 1 / (1 + np.exp(-z[t])), 0.0)
        else:
            score = np.where(live, np.exp(z[t] - z[t].max()), 0.0)
            score = score / score.sum()
        key = np.where(live, score + bias, -np.inf)
        if case["top_groups"] < case["groups"]:
            best = -np.sort(-key.reshape(-1, per), axis=1)[:, : case["group_top"]]
            total = np.where(best[:, 0] > -np.inf, np.where(best > -np.inf, best, 0).sum(1), -np.inf)
            chosen = np.argsort(-total, kind="stable")[: case["top_groups"]]
            inside = np.isin(np.arange(case["experts"]) // per, chosen)
            key = np.where(inside, key, -np.inf)
        order = np.argsort(-key, kind="stable")[: case["k"]]
        order = order[key[order] > -np.inf]
        w = score[order]
        if case["renorm"]:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        idx[t, : len(order)], wgt[t, : len(order)] = order, case["scale"] * w
    return idx, wgt
