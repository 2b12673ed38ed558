"""Attention over a paged key-value cache, in plain torch and as the framework's own calls: the quarter of the layers
that keeps a cache, beside the linear attention of the others.

  append   what a step's projections give enters the cache: per-head RMS norm of queries and keys, rotary positions on a
           part of each head, keys and values written into their sequence's pages, queries returned
  decode   attention of one new token for each sequence over its pages, grouped heads, sigmoid-gated outputs
  prefill  causal attention of several new tokens for each sequence (prompts, prompts that continue a cached
           conversation, drafted tokens), packed one after the other, over the same pages
"""
import math
import random

import torch

own = False

HEADS = dict(q_heads=16, kv_heads=2, dim=256)   # gated attention beside linear attention layers


# --------------------------------------------------------------------------- cases
# seqs: sequences; tokens: new tokens of all of them; ctx: the longest prefix that is cached before them
def listed():
    return [
        # one token of one sequence: latency
        dict(name="append_token", op="append", seqs=1, tokens=1, ctx=4095, **HEADS, page=64, norm=True, rot=64,
             act="bf16"),
        # the prompts of a batch, odd lengths
        dict(name="append_prompts", op="append", seqs=5, tokens=8191, ctx=1000, **HEADS, page=64, norm=True, rot=64,
             act="bf16"),
        # heads without norms, rotated whole, fp16, small pages
        dict(name="append_whole", op="append", seqs=3, tokens=701, ctx=33, q_heads=12, kv_heads=4, dim=128, page=16,
             norm=False, rot=128, act="f16"),
        # the first tokens of a conversation: latency
        dict(name="decode_first", op="decode", seqs=1, tokens=1, ctx=12, **HEADS, page=64, gate=True, act="bf16"),
        # one sequence at the far end of a long context
        dict(name="decode_long", op="decode", seqs=1, tokens=1, ctx=262142, **HEADS, page=64, gate=True, act="bf16"),
        # a decode batch of very different lengths
        dict(name="decode_batch", op="decode", seqs=64, tokens=64, ctx=8191, **HEADS, page=64, gate=True, act="bf16"),
        # smaller heads, three queries to a key head, small pages, no gates, fp16
        dict(name="decode_small", op="decode", seqs=7, tokens=7, ctx=1500, q_heads=12, kv_heads=4, dim=128, page=16,
             gate=False, act="f16"),
        # five drafted tokens
        dict(name="prefill_draft", op="prefill", seqs=1, tokens=5, ctx=4096, **HEADS, page=64, gate=True, act="bf16"),
        # a batch of prompts of very different lengths
        dict(name="prefill_prompts", op="prefill", seqs=12, tokens=6001, ctx=0, **HEADS, page=64, gate=True,
             act="bf16"),
        # one long prompt
        dict(name="prefill_long", op="prefill", seqs=1, tokens=8192, ctx=0, **HEADS, page=64, gate=True, act="bf16"),
        # conversations that go on: new turns over what is cached
        dict(name="prefill_turns", op="prefill", seqs=4, tokens=1023, ctx=12345, **HEADS, page=64, gate=True,
             act="bf16"),
        # a small layer: fp16, narrow heads, no gates
        dict(name="prefill_small", op="prefill", seqs=3, tokens=700, ctx=50, q_heads=6, kv_heads=2, dim=64, page=32,
             gate=False, act="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill"))
    dim = rng.choice((64, 128, 256))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    q_heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 8, 8, 16))
    case = dict(op=op, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 32, 64, 128, 256)),
                act=rng.choice(("bf16", "f16")))
    if op == "append":
        tokens = max(1, min(_log(rng, 1, 16384), 8191 * 20 * 256 // ((q_heads + 2 * kv_heads) * dim)))
        seqs = min(_log(rng, 1, 64), tokens)
        return dict(case, seqs=seqs, tokens=tokens, ctx=min(_log(rng, 1, 65536), 2 ** 19 // (seqs * kv_heads)),
                    norm=rng.random() < 0.6, rot=rng.choice((0, 16, dim // 4, dim // 2, dim)))
    case["gate"] = rng.random() < 0.5
    if op == "decode":
        seqs = _log(rng, 1, 256)
        ctx = min(_log(rng, 1, 262142), 262142 * 2 * 256 // (seqs * max(kv_heads, q_heads // 8) * dim))
        return dict(case, seqs=seqs, tokens=seqs, ctx=ctx)
    tokens, ctx = _log(rng, 1, 8192), rng.choice((0, _log(rng, 1, 32768)))
    # no more products, and no more room for the plain form's scores, than one prompt of 8192 tokens takes
    while (tokens + 2 * ctx) * tokens * q_heads > 8192 * 8192 * 16:
        tokens, ctx = max(1, tokens * 3 // 4), ctx * 3 // 4
    seqs = min(_log(rng, 1, 32), tokens)
    while seqs > 1 and seqs * max(tokens * q_heads, 8 * kv_heads * dim) * (tokens + ctx) > 8192 * 8192 * 16:
        seqs -= 1
    return dict(case, seqs=seqs, tokens=tokens, ctx=ctx)


_DT = {"bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-6


def _new(case):
    """New tokens of each sequence: one each for decode, else uneven; a batch of many holds a sequence without any."""
    n, total = case["seqs"], case["tokens"]
    if case["op"] == "decode":
        return [1] * n
    r = random.Random(n * 1000003 + total)
    cuts = sorted(int(total * r.random() ** 1.5) for _ in range(n - 1))
    if n > 2:
        cuts[1] = cuts[0]
    ends = [0] + cuts + [total]
    return [b - a for a, b in zip(ends, ends[1:])]


def _lengths(case):
    """Tokens of each sequence, the new ones included; the first has the longest prefix. A large decode batch holds a
    place that no sequence takes."""
    r = random.Random(case["seqs"] * 10007 + case["ctx"])
    old = [case["ctx"]] + [int(case["ctx"] * r.random()) for _ in range(case["seqs"] - 1)]
    total = [a + b for a, b in zip(old, _new(case))]
    if case["op"] == "decode" and len(total) > 2:
        total[2] = 0
    return total


# --------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt = _DT[case["act"]]

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    n, hq, hk, d, page = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    new, total = _new(case), _lengths(case)
    pages = [-(-t // page) for t in total]
    width = max(pages) + 1                       # room for tokens to come
    free = torch.randperm(sum(pages) + 1, generator=gen, device="cuda").int()
    table = torch.full((len(pages), width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda") < torch.tensor(pages, device="cuda").unsqueeze(1)
    table[at] = free[: sum(pages)]               # pages lie in no order
    shape = (sum(pages) + 1, hk, page, d)
    off = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    s = dict(k_cache=randn(*shape), v_cache=randn(*shape).add_(0.5 * randn(hk, 1, d)), table=table, off=off,
             lengths=torch.tensor(total, dtype=torch.int32, device="cuda"), new=new, total=total,
             scale=1.0 / math.sqrt(d))
    if case["op"] == "append":
        # one projection's output holds a token's queries, gates, keys and values
        rows = randn(n, (2 * hq + 2 * hk) * d)
        s["q"] = rows[:, : 2 * hq * d].view(n, hq, 2, d)[:, :, 0]
        s["k"], s["v"] = rows[:, 2 * hq * d :].view(n, 2, hk, d).unbind(1)
        s["q_norm"] = 1 + 0.2 * randn(d, dtype=torch.float32) if case["norm"] else None
        s["k_norm"] = 1 + 0.2 * randn(d, dtype=torch.float32) if case["norm"] else None
        pairs = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        s["freq"] = 1e7 ** (-2 * pairs / max(case["rot"], 1)) if case["rot"] else None
        return s
    rows = randn(n, hq, 2, d)                    # queries and gates as a projection gives them
    s["q"], s["gate"] = rows[:, :, 0].mul_(1.5), rows[:, :, 1] if case["gate"] else None
    return s


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if case["op"] == "append":
        s["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    else:
        s["o"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    if own:
        from int4_routed_expert_router_amd import api
        s["api"] = api
        s["cache"] = api.KVCache(s["k_cache"], s["v_cache"], s["table"], s["lengths"])
        if case["op"] != "append":
            s["ws"] = api.attn_workspace(s["cache"], case["q_heads"], case["tokens"])
    return s


# --------------------------------------------------------------------------- plain forms
def _tokens(s):
    """Sequence and position of every new token."""
    t = torch.arange(s["case"]["tokens"], dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(s["off"][1:].contiguous(), t, right=True)
    first = s["lengths"] - (s["off"][1:] - s["off"][:-1])
    return seq, (first[seq] + t - s["off"][seq]).long()


def _append_plain(s):
    c = s["case"]
    seq, pos = _tokens(s)

    def head(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * weight
        if not c["rot"]:
            return x
        angle = (pos.double().unsqueeze(1) * s["freq"]).unsqueeze(1)   # positions are far: angles in 64 bits
        cos, sin = angle.cos().float(), angle.sin().float()
        a, b, rest = x.split([c["rot"] // 2, c["rot"] // 2, c["dim"] - c["rot"]], -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)

    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    s["q_out"].copy_(head(s["q"], s["q_norm"]))
    s["k_cache"][page, :, slot] = head(s["k"], s["k_norm"]).to(s["k_cache"].dtype)
    s["v_cache"][page, :, slot] = s["v"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _gather(s, cache):
    """[B, kv heads, positions, d] of each sequence's pages in 32 bits; 0 behind its length."""
    x = cache[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)
    dead = torch.arange(x.shape[2], device="cuda") >= s["lengths"].unsqueeze(1)
    return x.float().masked_fill_(dead[:, None, :, None], 0.0), dead


def _attend(s, q, allowed):
    """softmax(scale q k^T) v for q [B, kv heads, rows, d] over the positions that allowed [B, rows, positions] leaves."""
    k, _ = _gather(s, s["k_cache"])
    p = q @ k.transpose(-1, -2).contiguous()
    del k
    p.mul_(s["scale"]).masked_fill_(~allowed.unsqueeze(1), float("-inf"))
    p.sub_(p.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    v, _ = _gather(s, s["v_cache"])
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _decode_plain(s):
    c = s["case"]
    q = s["q"].float().view(c["seqs"], c["kv_heads"], -1, c["dim"])
    live = torch.arange(s["table"].shape[1] * c["page"], device="cuda") < s["lengths"].unsqueeze(1)
    o = _attend(s, q, live.unsqueeze(1)).view(s["q"].shape)
    s["o"].copy_(o if s["gate"] is None else o * torch.sigmoid(s["gate"].float()))
    return s["o"]


def _prefill_plain(s):
    c = s["case"]
    rep, most = c["q_heads"] // c["kv_heads"], max(s["new"])
    seq, pos = _tokens(s)
    at = torch.arange(c["tokens"], device="cuda") - s["off"][seq]
    q = torch.zeros(c["seqs"], most, c["q_heads"], c["dim"], device="cuda")
    q[seq, at] = s["q"].float()                                # sequences padded to the longest
    q = q.view(c["seqs"], most, c["kv_heads"], rep, c["dim"]).permute(0, 2, 3, 1, 4).flatten(2, 3).contiguous()
    last = torch.full((c["seqs"], most), -1, dtype=torch.long, device="cuda")
    last[seq, at] = pos
    allowed = torch.arange(s["table"].shape[1] * c["page"], device="cuda") <= last.unsqueeze(-1)
    o = _attend(s, q, allowed.repeat(1, rep, 1))
    o = o.view(c["seqs"], c["kv_heads"], rep, most, c["dim"]).permute(0, 3, 1, 2, 4)[seq, at].reshape(s["q"].shape)
    s["o"].copy_(o if s["gate"] is None else o * torch.sigmoid(s["gate"].float()))
    return s["o"]


def run(s):
    c = s["case"]
    if not own:
        return {"append": _append_plain, "decode": _decode_plain, "prefill": _prefill_plain}[c["op"]](s)
    if c["op"] == "append":
        s["api"].kv_append(s["cache"], s["k"], s["v"], seq_off=s["off"], q=s["q"], q_out=s["q_out"],
                           q_norm=s["q_norm"], k_norm=s["k_norm"], eps=_EPS, freq=s["freq"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if c["op"] == "decode":
        s["api"].attn_decode(s["cache"], s["q"], s["o"], s["scale"], gate=s["gate"], ws=s["ws"])
    else:
        s["api"].attn_prefill(s["cache"], s["q"], s["o"], s["off"], s["scale"], gate=s["gate"], ws=s["ws"])
    return s["o"]


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    n, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        return {"bytes": 2 * 2 * n * (hq + 2 * hk) * d, "flops": n * (hq + hk) * (4 * d * case["norm"] + 3 * case["rot"])}
    new, total = _new(case), _lengths(case)
    if case["op"] == "decode":
        seen = sum(total)
    else:
        seen = sum(t * m - m * (m - 1) // 2 for m, t in zip(new, total))   # token i of m sees t - m + 1 + i
    live = sum(t for m, t in zip(new, total) if m)
    return {"bytes": 2 * n * hq * d * (3 if case["gate"] else 2) + 2 * 2 * live * hk * d, "flops": 4 * seen * hq * d}


# --------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        return _append_exact(case, s)
    rep, out = case["q_heads"] // case["kv_heads"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (m, t) in enumerate(zip(s["new"], s["total"])):
        if m == 0 or t == 0:
            continue
        pages, first = s["table"][b, : -(-t // case["page"])].long(), sum(s["new"][:b])
        for h in range(case["kv_heads"]):
            k = s["k_cache"][pages, h].reshape(-1, case["dim"])[:t].double()
            v = s["v_cache"][pages, h].reshape(-1, case["dim"])[:t].double()
            for g in range(h * rep, (h + 1) * rep):
                z = torch.mm(s["q"][first : first + m, g].double(), k.t()) * s["scale"]
                z.masked_fill_(torch.ones(m, t, dtype=torch.bool, device="cuda").triu_(t - m + 1), float("-inf"))
                out[first : first + m, g] = torch.mm(torch.softmax(z, -1), v)
    return out if s["gate"] is None else out / (1 + torch.exp(-s["gate"].double()))


def _append_exact(case, s):
    half, page = case["rot"] // 2, case["page"]
    pos = torch.cat([torch.arange(t - m, t) for m, t in zip(s["new"], s["total"])]).cuda()
    turn = None if not half else torch.polar(torch.ones(len(pos), half, dtype=torch.float64, device="cuda"),
                                             pos.double()[:, None] * s["freq"][None]).unsqueeze(1)

    def head(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + _EPS).sqrt() * weight.double()
        if turn is not None:   # pair (i, i + half) as one complex number
            z = torch.complex(x[..., :half].contiguous(), x[..., half : 2 * half].contiguous()) * turn
            x = torch.cat([z.real, z.imag, x[..., 2 * half :]], -1)
        return x

    k, v, kc, vc = head(s["k"], s["k_norm"]), s["v"].double(), s["k_cache"].double(), s["v_cache"].double()
    i = 0
    for b, (m, t) in enumerate(zip(s["new"], s["total"])):
        p = torch.arange(t - m, t, device="cuda")
        rows = s["table"][b, p // page].long()
        kc[rows, :, p % page], vc[rows, :, p % page] = k[i : i + m], v[i : i + m]
        i += m
    return head(s["q"], s["q_norm"]), kc, vc
