"""More tokens than a launch of the scored choice holds are refused before any
GPU work."""
import ctypes as C

import pytest

from int4_routed_expert_router_amd import api
from int4_routed_expert_router_amd._lib import lib


@pytest.mark.parametrize("T", [2 ** 26 - 3, 2 ** 31 - 4, 2 ** 31 - 1])
def test_too_many_tokens(T):
    sel = api.SelectDesc(16, 2)
    p = 4096
    assert lib().moe_select(sel.c(), p, 16, None, T, p, p, None, None) == -2
    assert b"n_tokens" in lib().moe_last_error()
    d, w = api.Desc(256, 16, 2, 64, 0, 32), api.Layer(p, None, p, 30720)
    assert lib().moe_route_scored(C.byref(d.c()), sel.c(), C.byref(w.c()), p, T, p, p, None, None, p, 1 << 62, None) == -2
    assert b"n_tokens" in lib().moe_last_error()
