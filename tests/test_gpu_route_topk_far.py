"""Chosen experts whose scores are 0 in 64 bits beside the others': bias or groups
keep the experts that dwarf them out.  Renormalized softmax weights are the softmax
over the chosen logits there, as everywhere, and so is their gradient; sigmoids
whose sum is 0 have weights 0 and no gradient.

Weights are 64-bit values rounded once to fp32; the tolerances are those of
test_gpu_route_topk."""

import numpy as np
import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

from .test_gpu_route_topk import check, check_gradient

pytestmark = pytest.mark.gpu

FAR = (-801.0, -5000.0, -3e38)


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("how", ["bias", "groups"])
def test_softmax_over_the_chosen(how, far):
    E, k = 64, 4
    g = torch.Generator().manual_seed(11)
    l = torch.zeros(6, E)
    l[:, :16] = torch.randn(6, 16, generator=g)  # what dwarfs the rest
    low = torch.randint(-8, 9, (6, 48), generator=g) * 2.0 ** -2
    l[:, 16:] = far + (low if far > -1e6 else 0.0)
    bias = torch.zeros(E)
    bias[:16] = -10.0
    opt = dict(scoring="softmax", scale=2.5)
    if how == "groups":  # the first group's bias leaves it behind the others
        opt.update(n_group=4, topk_group=2, group_top=2)
    ids, w = check(l, k, bias, **opt)
    assert (ids >= 16).all()
    x = l.gather(1, ids.cpu().long()).double()
    want = torch.softmax(x, 1) * 2.5
    assert ((w.cpu().double() - want).abs() <= (2.0 ** -24 + 1e-13) * want).all()
    assert (w.double().sum(1) - 2.5).abs().max() <= 4 * 2.0 ** -24 * 2.5
    # all equally: the lowest ids, since s + bias is the same for every one of them
    assert ids.tolist() == [[16, 17, 18, 19]] * 6


def test_sigmoids_that_vanish():
    l = torch.full((2, 32), -900.0)
    l[1, 3] = -600.0
    ids, w = check(l, 4, scoring="sigmoid", scale=2.5)
    assert not w[0].any() and ids[0].tolist() == [0, 1, 2, 3]
    assert ids[1].tolist() == [3, 0, 1, 2] and w[1].tolist() == [2.5, 0.0, 0.0, 0.0]
    d = moe.moe_route_topk_backward(l.cuda(), ids, torch.ones(2, 4, device="cuda"), "sigmoid", True, 2.5)
    assert not d[0].any()
    check_gradient(l, ids, "f32", "sigmoid", True, 2.5)


def test_not_renormalized():
    # the scores themselves: 0
    l = torch.zeros(1, 8)
    l[0, 4:] = -2000.0
    bias = torch.tensor([-9.0] * 4 + [0.0] * 4)
    ids, w = check(l, 2, bias, scoring="softmax", renormalize=False)
    assert ids.tolist() == [[4, 5]] and np.array_equal(w.cpu().numpy(), [[0.0, 0.0]])
