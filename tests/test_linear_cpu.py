"""The int4 linear product: sizes, refusals before any GPU work, and pins of
its oracle."""
import ctypes as C

import numpy as np
import pytest
import torch

from int4_routed_expert_router_amd import api
from int4_routed_expert_router_amd._lib import LinearDesc, lib
from oracle import linear_oracle as lo


def test_bytes():
    assert lib().moe_linear_bytes(2048, 8192, 64) == 8192 * 2048 // 2 + 4 * 8192 * 32
    assert lib().moe_linear_bytes(64, 1, 32) == 32 * 64 // 2 + 4 * 32 * 2     # padded to 32 rows
    assert lib().moe_linear_bytes(65536, 1 << 20, 128) == (1 << 20) * (32768 + 4 * 512)
    for bad in ((63, 1, 32), (96, 8, 32), (0, 8, 32), (65600, 8, 64), (64, 0, 32), (64, (1 << 20) + 1, 32),
                (64, 8, 48), (64, 8, 128), (64, -1, 64)):
        assert lib().moe_linear_bytes(*bad) == 0


def fwd(d=(64, 8, 64, 2, 3), packed=4096, x=4096, T=1, y=4096):
    st = lib().moe_linear_forward(C.byref(LinearDesc(*d)), packed, x, T, y, None)
    return st, lib().moe_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(d=(65, 8, 64, 2, 3)), -2), (dict(d=(64, 0, 64, 2, 3)), -2), (dict(d=(64, 8, 128, 2, 3)), -2),
    (dict(d=(64, 8, 64, 3, 3)), -1), (dict(d=(64, 8, 64, 0, 3)), -1), (dict(d=(64, 8, 64, 2, 0)), -1),
    (dict(d=(64, 8, 64, 2, 4)), -1), (dict(T=-1), -2), (dict(T=(1 << 20) + 1), -2), (dict(packed=None), -1),
    (dict(packed=4096 + 128), -1), (dict(x=None), -1), (dict(x=4096 + 8), -1), (dict(y=None), -1),
    (dict(y=4096 + 2), -1), (dict(d=(64, 8, 64, 2, 1), y=4096 + 1), -1)])
def test_forward_refusals(kw, status):
    assert fwd(**kw)[0] == status and fwd(**kw)[1]


def test_no_desc_and_no_tokens():
    assert lib().moe_linear_forward(None, 4096, 4096, 1, 4096, None) == -1
    assert fwd(T=0, packed=None, x=None, y=None) == (0, "")


def test_pack_refusals():
    def pack(K=64, N=8, G=64, q=4096, s=4096, b=4096, p=4096):
        return lib().moe_linear_pack(K, N, G, q, s, b, p, None)
    assert pack(K=32) == -2 and pack(N=0) == -2 and pack(G=16) == -2
    assert pack(q=None) == -1 and pack(s=None) == -1 and pack(b=None) == -1 and pack(p=None) == -1
    assert pack(q=4097) == -1 and pack(p=4096 + 64) == -1


def test_binding_refusals():
    w, s = torch.zeros(8, 8, dtype=torch.int32), torch.zeros(8, 1, dtype=torch.float16)
    with pytest.raises(ValueError, match="unsupported linear"):
        api.Linear(65, 8, 64, w, s, s)
    with pytest.raises(ValueError, match="act_dtype"):
        api.Linear(64, 8, 64, w, s, s, act_dtype="fp8")
    with pytest.raises(ValueError, match="words must be a CUDA tensor"):
        api.Linear(64, 8, 64, w, s, s)
    lin = api.Linear.__new__(api.Linear)
    lin.in_dim, lin.out_dim, lin.act_dtype, lin.packed = 64, 8, "bf16", torch.zeros(1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="y must be"):
        api.linear(lin, torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(1, 8, dtype=torch.float64))
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        api.linear(lin, torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(1, 8))


def test_oracle_pins():
    rng = np.random.default_rng(0)
    q = rng.integers(0, 16, (5, 128))
    assert np.array_equal(lo.unpack_words(lo.pack_words(q)), q)
    # a unit vector reads one weight: s q + b
    x = np.zeros((1, 128))
    x[0, 70] = 1.0
    s, b = rng.standard_normal((5, 4)), rng.standard_normal((5, 4))
    np.testing.assert_allclose(lo.linear(x, q, s, b, 32)[0], s[:, 2] * q[:, 70] + b[:, 2], rtol=1e-15)
    # agrees with the dequantisation of the layer's oracle
    from oracle import moe_oracle as mo
    sb = s.astype(np.float16)
    bb = b.astype(np.float16)
    w = mo.dequant(q.astype(np.uint8), sb.view(np.uint16), bb.view(np.uint16), 32)
    x = rng.standard_normal((3, 128))
    np.testing.assert_allclose(lo.linear(x, q, sb, bb, 32), x @ w.T, rtol=1e-12)
