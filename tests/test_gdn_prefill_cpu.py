"""moe_gdn_prefill refuses bad sizes, pointers, workspaces and tensors before
any GPU work; the sequence oracle agrees with chained steps."""
import ctypes as C

import numpy as np
import pytest
import torch

from int4_routed_expert_router_amd import api
from int4_routed_expert_router_amd._lib import GdnDesc, lib
from oracle import deltanet_oracle as dn

GOOD = (2, 16, 32, 128, 128, 2)


def call(desc=GOOD, N=100, ws_bytes=None, **ptr):
    p = dict(off=4096, q=4096, k=4096, v=4096, g=4096, beta=4096, state=4096, o=4096, ws=4096)
    p.update(ptr)
    d = GdnDesc(*desc)
    if ws_bytes is None:
        n = C.c_size_t(0)
        lib().moe_gdn_prefill_workspace_bytes(C.byref(d), max(N, 0), C.byref(n))
        ws_bytes = n.value
    st = lib().moe_gdn_prefill(C.byref(d), p["off"], N, p["q"], p["k"], p["v"], p["g"], p["beta"], 1.0, p["state"],
                               p["o"], p["ws"], ws_bytes, None)
    return st, lib().moe_last_error().decode()


@pytest.mark.parametrize("desc", [(-1, 1, 1, 128, 16, 2), (65536, 1, 1, 128, 16, 2), (1, 0, 1, 128, 16, 2),
                                  (1, 2, 3, 128, 16, 2), (1, 1, 1025, 128, 16, 2), (1, 1, 1, 64, 16, 2),
                                  (1, 1, 1, 128, 8, 2), (1, 1, 1, 128, 24, 2), (1, 1, 1, 128, 272, 2)])
def test_bad_shapes(desc):
    st, msg = call(desc, ws_bytes=1 << 30)
    assert st == -2 and msg
    n = C.c_size_t(0)
    assert lib().moe_gdn_prefill_workspace_bytes(C.byref(GdnDesc(*desc)), 5, C.byref(n)) == -2


def test_bad_arguments():
    assert call((1, 1, 1, 128, 16, 3))[0] == -1
    assert call(N=-1)[0] == -2 and call(N=(1 << 30) + 1, ws_bytes=1 << 40)[0] == -2
    for name in ("off", "q", "k", "v", "g", "beta", "state", "o", "ws"):
        assert call(**{name: None})[0] == -1
    for name, p in (("q", 4096 + 8), ("k", 4096 + 8), ("v", 4097), ("state", 4096 + 8), ("off", 4098), ("g", 4098),
                    ("beta", 4098), ("o", 4098), ("ws", 4096 + 128)):
        assert call(**{name: p})[0] == -1
    assert call(ws_bytes=255)[0] == -3
    assert lib().moe_gdn_prefill(None, 4096, 1, *[4096] * 5, 1.0, 4096, 4096, 4096, 1 << 30, None) == -1
    assert lib().moe_gdn_prefill_workspace_bytes(C.byref(GdnDesc(*GOOD)), 5, None) == -1


def test_nothing_to_do():
    none = dict(off=None, q=None, k=None, v=None, g=None, beta=None, state=None, o=None, ws=None)
    assert call(N=0, **none) == (0, "")
    assert call((0, 16, 32, 128, 128, 2), **none) == (0, "")


def test_workspace_grows_with_the_call():
    def size(B, N, hk=16, hv=32, dv=128):
        n = C.c_size_t(0)
        assert lib().moe_gdn_prefill_workspace_bytes(C.byref(GdnDesc(B, hk, hv, 128, dv, 2)), N, C.byref(n)) == 0
        return n.value
    assert size(1, 0) <= size(1, 64) <= size(1, 65) <= size(1, 8192) <= size(8, 8192) <= size(8, 8192, 16, 64)


def test_binding_refusals():
    f, h = torch.float32, torch.bfloat16
    q, v = torch.zeros(5, 2, 128, dtype=h), torch.zeros(5, 4, 16, dtype=h)
    g, st, o, off = torch.zeros(5, 4), torch.zeros(1, 4, 16, 128), torch.zeros(5, 4, 16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        api.gdn_prefill(q, q, v, g, g, st, o, off, 1.0)
    with pytest.raises(ValueError, match="dimensions"):
        api.gdn_prefill(q[0], q, v, g, g, st, o, off, 1.0)
    assert f == st.dtype


def test_sequence_oracle_is_the_step_chained():
    rng = np.random.default_rng(0)
    lens, Hk, Hv, dv = [3, 0, 2], 1, 2, 16
    N = sum(lens)
    q, k, v = rng.standard_normal((N, Hk, 128)), rng.standard_normal((N, Hk, 128)), rng.standard_normal((N, Hv, dv))
    g, beta = -rng.random((N, Hv)), rng.random((N, Hv))
    s0 = rng.standard_normal((3, Hv, dv, 128))
    S, o = dn.gdn_sequences(s0, q, k, v, g, beta, 0.3, lens)
    s = s0[2:3]
    for t in (3, 4):
        s, ot = dn.gdn_step(s, q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], beta[t:t + 1], 0.3)
        np.testing.assert_array_equal(ot[0], o[t])
    np.testing.assert_array_equal(s[0], S[2])
    np.testing.assert_array_equal(s0[1], S[1])
