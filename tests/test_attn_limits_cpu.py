"""Refusals of the paged attention calls at the ends of their ranges, before any GPU work."""
import pytest

from int4_routed_expert_router_amd._lib import lib
from test_attn_cpu import attend


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("scale", [3e38, -3e38, 2.0 ** 127.5])
def test_scales_that_leave_fp32_in_powers_of_two(which, scale):
    # the kernels take scale * log2(e): infinity times a score of 0 is no score
    assert attend(which, scale=scale) == -1
    assert b"scale" in lib().moe_last_error()
