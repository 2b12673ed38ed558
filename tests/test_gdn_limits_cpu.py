"""Sizes of moe_gdn_prefill that no launch can hold are refused before any GPU
work, by the call and by its workspace's size alike."""
import ctypes as C

import pytest

from int4_routed_expert_router_amd._lib import GdnDesc, lib


@pytest.mark.parametrize("B,N,ok", [(1, 1 << 30, False), (63, (1 << 30) - 64 * 64, True), (64, (1 << 30) - 64 * 64, False),
                                    (65535, (1 << 30) - 64 * 65536, True), (65535, (1 << 30) - 64 * 65535, False)])
def test_more_blocks_than_a_grid_holds(B, N, ok):
    d, n = GdnDesc(B, 1, 1, 128, 16, 2), C.c_size_t(0)
    assert lib().moe_gdn_prefill_workspace_bytes(C.byref(d), N, C.byref(n)) == (0 if ok else -2)
    if ok:
        assert n.value > 0
        return
    assert b"2^24" in lib().moe_last_error()
    p = 4096
    assert lib().moe_gdn_prefill(C.byref(d), p, N, p, p, p, p, p, 1.0, p, p, p, 1 << 62, None) == -2
