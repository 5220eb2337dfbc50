"""Pins of the general router's oracle (CPU only)."""

import math

import numpy as np
import pytest

from oracle.route_topk import route_topk_backward_ref, route_topk_ref, scores
from oracle.router import route_ref


def test_hand_case():
    # logits ln(1), ln(2), ln(3), ln(4): softmax 0.1 .. 0.4
    l = np.log(np.array([[1.0, 2, 3, 4]]))
    ids, w = route_topk_ref(l, 2)
    assert ids.tolist() == [[3, 2]] and np.allclose(w, [[4 / 7, 3 / 7]], rtol=1e-12)
    # the bias chooses, the weights stay the scores
    ids, w = route_topk_ref(l, 2, bias=[1, 0, 0, 0], renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 3]] and np.allclose(w, [[0.2, 0.8]], rtol=1e-12)
    # groups (0, 1), (2, 3) by the sum of two: 0.3 against 0.7; with a bias of 0.5 on 0: 0.8
    assert route_topk_ref(l, 1, n_group=2, topk_group=1, group_top=2)[0].tolist() == [[3]]
    assert route_topk_ref(l, 2, bias=[0.5, 0, 0, 0], n_group=2, topk_group=1, group_top=2)[0].tolist() == [[0, 1]]
    # sigmoid of ln a is a / (1 + a)
    assert np.allclose(scores(l, "sigmoid"), [[1 / 2, 2 / 3, 3 / 4, 4 / 5]], rtol=1e-12)


def test_masks_and_ties():
    inf, nan = math.inf, math.nan
    ids, w = route_topk_ref([[-inf, 0.0, nan, -inf], [-inf] * 4, [1.0, 1, 1, 1]], 2)
    assert ids.tolist() == [[1, -1], [-1, -1], [0, 1]]
    assert w.tolist() == [[1, 0], [0, 0], [0.5, 0.5]]
    # a group of masked experts is not kept, whatever the others' sums
    ids, _ = route_topk_ref([[-inf, -inf, -9.0, -9.0]], 2, scoring="sigmoid", bias=[0, 0, -5, -5.0], n_group=2,
                            topk_group=1, group_top=2)
    assert ids.tolist() == [[2, 3]]


def test_plain_router_is_a_special_case():
    l = np.random.default_rng(3).normal(size=(50, 24))
    ids, w = route_topk_ref(l, 4)
    ref_ids, ref_w = route_ref(l, 4)
    assert np.array_equal(ids, ref_ids) and np.allclose(w, ref_w, rtol=1e-12)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_by_differences(scoring, renorm):
    rng = np.random.default_rng(7)
    l, dw = rng.normal(size=(3, 10)), rng.normal(size=(3, 4))
    args = dict(scoring=scoring, renormalize=renorm, scale=1.5)
    ids, _ = route_topk_ref(l, 4, bias=rng.normal(size=10), **args)
    from oracle.route_topk import chosen_weights
    got, h = route_topk_backward_ref(l, ids, dw, scoring, renorm, 1.5), 1e-5
    for t in range(3):
        for e in range(10):
            d = np.zeros_like(l)
            d[t, e] = h
            num = ((chosen_weights(l + d, ids, **args) - chosen_weights(l - d, ids, **args)) * dw).sum() / (2 * h)
            assert abs(got[t, e] - num) < 1e-8
