"""The paged attention calls refuse bad sizes, pointers, strides, workspaces and
tensors before any GPU work; the attention oracle in closed forms."""
import ctypes as C

import numpy as np
import pytest
import torch

from int4_routed_expert_router_amd import api
from int4_routed_expert_router_amd._lib import AttnDesc, AttnRows, KvCacheC, lib
from oracle import attention_oracle as ao

# batch, q_heads, kv_heads, head_dim, act, page_size, n_pages, max_pages
GOOD = (2, 16, 2, 256, 2, 64, 10, 4)


def need(desc, n):
    b = C.c_size_t(0)
    st = lib().moe_attn_workspace_bytes(C.byref(AttnDesc(*desc)), n, C.byref(b))
    return st, b.value


def rows(p=4096, st=4096, sh=256):
    return AttnRows(p, st, sh)


def ref(x):
    return None if x is None else C.byref(x)


def attend(which, desc=GOOD, N=5, cache=(4096,) * 4, off=4096, q=(4096, 4096, 256), gate=None, scale=1.0, o=4096,
           ws=4096, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = need(desc, max(N, 0))[1]
    c = None if cache is None else KvCacheC(*cache)
    q, g = (None if r is None else rows(*r) for r in (q, gate))
    d = AttnDesc(*desc)
    if which == "decode":
        return lib().moe_attn_decode(C.byref(d), ref(c), ref(q), ref(g), scale, o, ws, ws_bytes, None)
    return lib().moe_attn_prefill(C.byref(d), ref(c), off, N, ref(q), ref(g), scale, o, ws, ws_bytes, None)


def append(desc=GOOD, N=5, cache=(4096,) * 4, off=4096, k=(4096, 4096, 256), v=(4096, 4096, 256), q=(4096, 4096, 256),
           q_out=4096, q_norm=None, k_norm=None, eps=1e-6, freq=4096, rot=64):
    c = None if cache is None else KvCacheC(*cache)
    k, v, q = (None if r is None else rows(*r) for r in (k, v, q))
    return lib().moe_kv_append(C.byref(AttnDesc(*desc)), ref(c), off, N, ref(k), ref(v), ref(q), q_out, q_norm, k_norm,
                               eps, freq, rot, None)


BAD_SHAPES = [(-1, 16, 2, 256, 2, 64, 10, 4), (65536, 16, 2, 256, 2, 64, 10, 4), (2, 16, 0, 256, 2, 64, 10, 4),
              (2, 129, 129, 256, 2, 64, 10, 4), (2, 1, 2, 256, 2, 64, 10, 4), (2, 3, 2, 256, 2, 64, 10, 4),
              (2, 34, 2, 256, 2, 64, 10, 4), (2, 16, 2, 96, 2, 64, 10, 4), (2, 16, 2, 512, 2, 64, 10, 4),
              (2, 16, 2, 256, 2, 8, 10, 4), (2, 16, 2, 256, 2, 48, 10, 4), (2, 16, 2, 256, 2, 512, 10, 4),
              (2, 16, 2, 256, 2, 64, 0, 4), (2, 16, 2, 256, 2, 64, 10, 0), (2, 16, 2, 256, 2, 64, 10, 1 << 25),
              (65535, 16, 2, 256, 2, 256, 10, 1 << 22)]


@pytest.mark.parametrize("desc", BAD_SHAPES, ids=str)
def test_bad_shapes(desc):
    assert need(desc, 5)[0] == -2
    for which in ("decode", "prefill"):
        assert attend(which, desc, ws_bytes=1 << 40) == -2 and lib().moe_last_error()
    assert append(desc) == -2


def test_bad_arguments():
    wrong = GOOD[:4] + (3,) + GOOD[5:]
    assert need(wrong, 5)[0] == -1 and append(wrong) == -1
    assert lib().moe_attn_workspace_bytes(C.byref(AttnDesc(*GOOD)), 5, None) == -1
    assert lib().moe_attn_workspace_bytes(None, 5, None) == -1
    for n in (-1, (1 << 20) + 1):
        assert need(GOOD, n)[0] == -2 and append(N=n) == -2 and attend("prefill", N=n, ws_bytes=1 << 40) == -2
    for which in ("decode", "prefill"):
        assert attend(which, cache=None) == -1 and attend(which, q=None) == -1
        for i, p in ((0, None), (1, None), (2, None), (3, None), (0, 4104), (1, 4104), (2, 4098), (3, 4098)):
            cache = [4096] * 4
            cache[i] = p
            assert attend(which, cache=cache) == -1
        for r in ((None, 256, 256), (4104, 256, 256)):
            assert attend(which, q=r) == -1 and attend(which, gate=r) == -1
        for r in ((4096, 4, 256), (4096, 256, 4), (4096, -256, 256), (4096, 256, -8), (4096, 1 << 37, 8)):
            assert attend(which, q=r) == -2 and attend(which, gate=r) == -2
        for s in (float("inf"), float("nan")):
            assert attend(which, scale=s) == -1
        for p in (None, 4104):
            assert attend(which, o=p) == -1
        for p in (None, 4096 + 128):
            assert attend(which, ws=p) == -1
        assert attend(which, ws_bytes=255) == -3
    for p in (None, 4098):
        assert attend("prefill", off=p) == -1


def test_bad_append_arguments():
    assert append(cache=None) == -1 and append(k=None) == -1 and append(v=None) == -1
    assert append(off=None, N=5) == -2 and append(off=4098) == -1
    for rot in (-16, 8, 24, 272):
        assert append(rot=rot) == -2
    assert append(freq=None) == -1 and append(freq=4100) == -1
    assert append(q_out=None) == -1 and append(q_out=4104) == -1
    assert append(q=None) == -1 and append(q=None, q_out=None, q_norm=4096) == -1
    assert append(q_norm=4104) == -1 and append(k_norm=4104) == -1
    for eps in (-1.0, float("nan"), float("inf")):
        assert append(k_norm=4096, eps=eps) == -1
    for r in ((4104, 256, 256), (None, 256, 256)):
        assert append(k=r) == -1 and append(v=r) == -1 and append(q=r) == -1
    for r in ((4096, 4, 256), (4096, 256, -8)):
        assert append(k=r) == -2 and append(v=r) == -2 and append(q=r) == -2


def test_nothing_to_do():
    empty = (0,) + GOOD[1:]
    for which in ("decode", "prefill"):
        assert attend(which, empty, cache=None, off=None, q=None, o=None, ws=None, ws_bytes=0) == 0
    assert attend("prefill", N=0, cache=None, off=None, q=None, o=None, ws=None, ws_bytes=0) == 0
    assert append(empty, N=0, cache=None, off=None, k=None, v=None, q=None, q_out=None, freq=None) == 0
    assert append(N=0, cache=None, off=4096, k=None, v=None, q=None, q_out=None, freq=None) == 0


@pytest.mark.parametrize("n,ok", [(1 << 20, False), (100000, True), (1 << 18, True), (300000, False)])
def test_more_units_than_a_grid_holds(n, ok):
    # 16 tokens to a unit: kv_heads (n / 16 + min(batch, n)) up to 2^22
    desc = (16384, 2048, 128, 64, 2, 16, 10, 1)
    assert need(desc, n)[0] == (0 if ok else -2)
    if not ok:
        assert b"launch" in lib().moe_last_error()
        assert attend("prefill", desc, N=n, ws_bytes=1 << 50) == -2


def test_workspace_covers_both_calls():
    assert need(GOOD, 0)[0] == 0 and need(GOOD, 0)[1] >= 256
    assert need(GOOD, 0)[1] <= need(GOOD, 5000)[1] <= need(GOOD, 1 << 20)[1] <= 1 << 30


def test_binding_refusals():
    bf = torch.bfloat16
    k = torch.zeros(4, 2, 16, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.KVCache(k, k, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="torch tensor"):
        api.KVCache(4096, k, None, None)


def test_oracle_closed_forms():
    rng = np.random.default_rng(3)
    page, hk, d, B = 16, 2, 8, 3
    table = np.array([[4, 1, -1], [0, 5, 2], [9, 3, -7]])        # page 9 is none
    length, off = np.array([20, 40, 30]), np.array([0, 3, 3, 5])
    kc, vc = rng.standard_normal((6, hk, page, d)), rng.standard_normal((6, hk, page, d))
    q = rng.standard_normal((6, 2 * hk, d))
    # a scale of 0: the mean of the values that the token sees
    o, bound = ao.attend(kc, vc, table, length, off, q, 0.0)
    rows0 = [vc[4, 1, s] for s in range(16)] + [vc[1, 1, s] for s in range(3)]
    np.testing.assert_allclose(o[1, 3], np.mean(rows0, 0))       # position 18 of sequence 0
    # sequence 2 lacks its first 16 positions
    np.testing.assert_allclose(o[4, 0], np.mean([vc[3, 0, s] for s in range(14)], 0))
    assert np.isnan(o[5]).all() and np.isnan(bound[5]).all() and (bound[:5] >= 0).all()
    # a large scale: the value of the largest score
    o, _ = ao.attend(kc, vc, table, length, off, q, 1e6)
    z = [kc[4, 0, s] @ q[0, 1] for s in range(16)] + [kc[1, 0, s] @ q[0, 1] for s in range(2)]
    best = int(np.argmax(z))
    np.testing.assert_allclose(o[0, 1], vc[4, 0, best] if best < 16 else vc[1, 0, best - 16])
    # a gate of 0 halves
    np.testing.assert_allclose(ao.attend(kc, vc, table, length, off, q, 1e6, gate=np.zeros_like(q))[0][:5], o[:5] / 2)
    # rotation keeps lengths and depends on distances only; norms give unit mean squares
    freq = np.array([1.0, 0.1])
    x, y = rng.standard_normal((2, 1, 4))
    turned = [[ao._head(a, None, 0, freq, p) for p in (5, 105)] for a in (x, y)]
    np.testing.assert_allclose((turned[0][0] * turned[1][0]).sum(), (turned[0][1] * turned[1][1]).sum())
    np.testing.assert_allclose((turned[0][1] ** 2).sum(), (x ** 2).sum())
    np.testing.assert_allclose((ao._head(x, np.full(4, 3.0), 0.0, None, 0) ** 2).mean(), 9.0)
    new = rng.standard_normal((6, hk, d))
    qo, k2, v2 = ao.append(kc, vc, table, length, off, new, new, q)
    assert np.array_equal(v2[1, :, 1], new[0]) and np.array_equal(v2[3, :, 13], new[4]) and np.isnan(qo[5]).all()
    assert (v2 != vc).any(-1).sum() == 5 * hk and np.array_equal(k2[v2 == vc], kc[v2 == vc])


def test_oracle_rows_of_short_sequences():
    assert ao.rows_of([5, -3, 99], [0, 2, 3, 4], 32) == [(0, 0, 3), (1, 0, 4), (2, 1, -1), (3, 2, 31)]
    assert ao.rows_of([5, 0], None, 32) == [(0, 0, 4), (1, 1, -1)]
