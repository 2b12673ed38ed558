"""Refusals of the paged attention calls at the ends of their ranges, before any GPU work."""
import os
import re

import pytest

from int4_routed_expert_router_amd._lib import lib
from test_attn_cpu import attend


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("scale", [3e38, -3e38, 2.0 ** 127.5])
def test_scales_that_leave_fp32_in_powers_of_two(which, scale):
    # the kernels take scale * log2(e): infinity times a score of 0 is no score
    assert attend(which, scale=scale) == -1
    assert b"scale" in lib().moe_last_error()


def test_assembly_names_what_it_overwrites():
    # the compiler keeps values of its own in m0, and its own waits do not reach into the statements
    from int4_routed_expert_router_amd import build
    found = 0
    for path in build.sources():
        for text in re.findall(r"asm volatile\((.*?)\);", open(path).read(), re.S):
            if "s_mov_b32 m0" not in text:
                continue
            found += 1
            template, *operands = text.split(":")
            assert '"m0"' in operands[-1], (os.path.basename(path), text)
            waits = 1 + sum(int(n) + 1 for n in re.findall(r"s_nop (\d+)", template))
            assert waits >= (2 if ", off" in template else 5), (os.path.basename(path), text)
    assert found == 2
