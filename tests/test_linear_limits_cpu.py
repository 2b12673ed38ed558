"""Linear products whose outputs no launch can hold are refused before any GPU
work (2^37 outputs: 256 GB in 16 bits)."""
import ctypes as C

import pytest

from int4_routed_expert_router_amd._lib import LinearDesc, lib


@pytest.mark.parametrize("T,N", [(1 << 20, 1 << 17), (1 << 17, 1 << 20), (1 << 20, (1 << 17) - 127), (1 << 20, 1 << 20)])
def test_more_tiles_than_a_grid_holds(T, N):
    d = LinearDesc(64, N, 64, 2, 1)
    assert lib().moe_linear_forward(C.byref(d), 4096, 4096, T, 4096, None) == -2
    assert b"tiles" in lib().moe_last_error()


def test_fewer_are_not():
    # without buffers: the next check answers
    d = LinearDesc(64, (1 << 17) - 128, 64, 2, 1)
    assert lib().moe_linear_forward(C.byref(d), None, None, 1 << 20, None, None) == -1
