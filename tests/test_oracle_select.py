"""Pins of the scored-choice oracle: closed forms, the equality with the plain
softmax top-K of the layer oracle, hand-made group cases."""
import math

import numpy as np

from oracle import moe_oracle as mo
from oracle import select_oracle as so


def test_softmax_renormalised_equals_the_layer_oracles_routing():
    z = np.random.default_rng(0).standard_normal((20, 33))
    idx, w = so.select(z, 6, "softmax")
    for t in range(20):
        ref = mo.topk_order(z[t], 6)
        assert idx[t].tolist() == ref.tolist()
        np.testing.assert_allclose(w[t], mo.renormalised_weights(z[t, ref]), rtol=1e-14)


def test_sigmoid_closed_forms():
    # sigmoid(ln 3) = 3/4, sigmoid(0) = 1/2, sigmoid(-ln 3) = 1/4
    idx, w = so.select_token([-math.log(3), 0.0, math.log(3)], 3, "sigmoid", renorm=False, scale=4.0)
    assert idx == [2, 1, 0]
    np.testing.assert_allclose(w, [3.0, 2.0, 1.0], rtol=1e-15)
    _, w = so.select_token([-math.log(3), 0.0, math.log(3)], 3, "sigmoid")
    np.testing.assert_allclose(w, [0.5, 1 / 3, 1 / 6], rtol=1e-15)


def test_bias_enters_the_choice_only():
    idx, w = so.select_token([0.0, 0.0, 0.0], 1, "sigmoid", bias=[0.0, 0.25, 0.0], renorm=False)
    assert idx == [1] and w == [0.5]
    idx, _ = so.select_token([0.0, 0.0, 0.0], 2, "sigmoid", bias=[0.0, 0.0, 0.0])
    assert idx == [0, 1]


def test_groups_by_their_two_best_keys():
    # group 0 holds the best expert, group 1 the best pair
    z = [3.0, -5.0, 2.0, 2.0]
    assert so.select_token(z, 2, "sigmoid", n_group=2, top_groups=1, group_top=2)[0] == [2, 3]
    assert so.select_token(z, 2, "sigmoid", n_group=2, top_groups=1, group_top=1)[0] == [0, 1]
    assert so.select_token(z, 2, "sigmoid", n_group=2, top_groups=2)[0] == [0, 2]


def test_experts_that_are_off():
    ninf = -math.inf
    assert so.select_token([ninf, 1.0, math.nan], 3, "softmax") == ([1, -1, -1], [1.0, 0.0, 0.0])
    assert so.select_token([ninf, ninf], 2, "sigmoid") == ([-1, -1], [0.0, 0.0])
    assert so.select_token([math.inf, 1.0, math.inf], 2, "softmax") == ([0, 2], [0.5, 0.5])
    # all scores 0: chosen by index, weight 0 after renormalisation of a zero sum
    assert so.select_token([-1e30, -2e30], 2, "sigmoid") == ([0, 1], [0.0, 0.0])
