"""GPU paged attention at the limits of its contract: rows that see nothing, scores and values near the ends of fp32's
range, scales of 0 and subnormal ones, tiny rows under a norm, sequences that take no part."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def case(*a, **k):
    from attn_testlib import Case
    return Case(*a, **k)


def same_bits(a, b):
    import torch
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_gates_of_rows_that_see_nothing(decode, value):
    # no positions, or pages that are none: 0 whatever the gate is; the other rows do not change
    new, total = ([1] * 4, [200, 0, 90, 40]) if decode else ([9, 0, 30, 40], [200, 0, 90, 33])
    c = case(new, total, 6, 2, 64, 16, "bf16", gate=True, seed=31)
    c.table[2, :] = -1
    none = [1, 2] if decode else list(range(9, 39)) + list(range(39, 46))   # of the last sequence 7 rows lie before it
    want = c.run(decode)
    c.check(want, decode)
    c.gate[none] = value
    o = c.run(decode)
    assert same_bits(o, want) and not o[none].any()


@pytest.mark.parametrize("act,d", [("bf16", 64), ("f16", 128), ("bf16", 256)])
def test_gates_of_rows_before_a_cut_unit(act, d):
    # one query to a key head: 256 tokens to a unit, whose tiles lie in several runs, its first ten rows at no position
    c = case([300], [290], 2, 2, d, 16, act, gate=True, seed=32)
    want = c.run()
    c.check(want)
    c.gate[:10] = float("nan")
    for _ in range(5):
        assert same_bits(c.run(), want)
