"""The scored choice refuses bad descriptors, sizes and tensors before any GPU
work (library and binding)."""
import ctypes as C
import dataclasses

import pytest
import torch

from int4_routed_expert_router_amd import MoeError, api
from int4_routed_expert_router_amd._lib import lib

GOOD = api.SelectDesc(256, 8, "sigmoid", 8, 4, 2)


def call(desc, logits=4096, stride=None, T=1, idx=8192, w=8192, gate=None):
    st = lib().moe_select(desc.c(), logits, desc.n_experts if stride is None else stride, None, T, idx, w, gate, None)
    return st, lib().moe_last_error().decode()


@pytest.mark.parametrize("change,status,word", [
    (dict(n_experts=0), -2, "n_experts"), (dict(n_experts=1025), -2, "n_experts"), (dict(top_k=0), -2, "top_k"),
    (dict(top_k=65), -2, "top_k"), (dict(n_experts=4, n_group=1, top_groups=1, top_k=5), -2, "top_k"),
    (dict(score="tanh"), -1, "score"), (dict(n_group=7), -2, "n_group"), (dict(n_group=128), -2, "n_group"),
    (dict(n_group=-8), -2, "n_group"), (dict(top_groups=9), -2, "top_groups"), (dict(top_groups=-1), -2, "top_groups"),
    (dict(n_experts=16, n_group=8, top_groups=3), -2, "top_groups"), (dict(group_top=3), -1, "group_top"),
    (dict(renorm=2), -1, "renorm"), (dict(scale=float("inf")), -1, "scale"), (dict(scale=float("nan")), -1, "scale"),
], ids=lambda v: str(v) if isinstance(v, dict) else "")
def test_bad_descriptors(change, status, word):
    st, msg = call(dataclasses.replace(GOOD, **change))
    assert st == status and word in msg


def test_bad_arguments():
    assert call(GOOD, stride=255)[0] == -2
    assert call(GOOD, stride=256, gate=4096)[0] == -2      # the gate is column E
    assert call(GOOD, T=-1)[0] == -2
    for missing in ("logits", "idx", "w"):
        assert call(GOOD, **{missing: None})[0] == -1
    assert lib().moe_select(None, 4096, 256, None, 1, 4096, 4096, None, None) == -1
    assert call(GOOD, T=0, logits=None, idx=None, w=None) == (0, "")
    # zeros read as defaults
    assert call(dataclasses.replace(GOOD, n_group=0, top_groups=0, group_top=0), T=0)[0] == 0


def test_route_scored_needs_matching_descriptors():
    d = api.Desc(256, 16, 2, 64, 0, 32)
    w = api.Layer(4096, None, 4096, 30720)
    for sel in (api.SelectDesc(16, 3), api.SelectDesc(32, 2)):
        with pytest.raises(MoeError, match="differs from the layer"):
            st = lib().moe_route_scored(C.byref(d.c()), sel.c(), C.byref(w.c()), 4096, 1, 4096, 4096, None, None, 4096,
                                        1 << 20, None)
            api.check(st)
    sel = api.SelectDesc(16, 2)
    args = (C.byref(d.c()), sel.c(), C.byref(w.c()))
    assert lib().moe_route_scored(*args, None, 1, 4096, 4096, None, None, 4096, 1 << 20, None) == -1
    assert lib().moe_route_scored(*args, 4096, 1, None, 4096, None, None, 4096, 1 << 20, None) == -1
    assert lib().moe_route_scored(*args, 4096, 1, 4096, 4096, None, None, 4096, 16, None) == -3
    assert lib().moe_route_scored(*args, None, 0, None, None, None, None, None, 0, None) == 0


def test_binding_refuses_host_and_misshaped_tensors():
    z, i, w = torch.zeros(3, 256), torch.zeros(3, 8, dtype=torch.int32), torch.zeros(3, 8)
    with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
        api.select(GOOD, z, i, w)
    with pytest.raises(ValueError, match="columns"):
        api.select(GOOD, torch.zeros(3, 255), i, w)
    with pytest.raises(ValueError, match=r"\[T, E\]"):
        api.select(GOOD, torch.zeros(256), i, w)
