"""Refusals of the general router (CPU only): the C entries reject bad
arguments before anything is enqueued, the binding rejects tensors that the
kernels do not take."""

import ctypes
import math

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

from .test_rows_abi_cpu import Fake as Face

P = ctypes.c_void_p
F, ODD = P(1 << 20), P((1 << 20) + 8)
NULL, SHAPE, UNSUPPORTED, ALIGN = -1, -2, -3, -4


class Fake(Face):
    requires_grad = False


def route(elem=2, logits=F, bias=None, T=4, E=16, k=2, scoring=0, groups=1, kept=1, top=1, renorm=1, scale=1.0,
          ids=F, w=F):
    return moe.lib().moe_route_topk(elem, logits, bias, T, E, k, scoring, groups, kept, top, renorm, scale, ids, w, None)


def backward(elem=2, logits=F, ids=F, dw=F, T=4, E=16, k=2, scoring=0, renorm=1, scale=1.0, d=F):
    return moe.lib().moe_route_topk_backward(elem, logits, ids, dw, T, E, k, scoring, renorm, scale, d, None)


@pytest.mark.parametrize("call", [route, backward])
@pytest.mark.parametrize("bad,status", [
    (dict(elem=3), UNSUPPORTED), (dict(elem=-1), UNSUPPORTED), (dict(scoring=2), UNSUPPORTED), (dict(T=-1), SHAPE),
    (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(E=1025), UNSUPPORTED), (dict(E=32, k=17), UNSUPPORTED),
    (dict(k=17), UNSUPPORTED), (dict(E=4, k=5), UNSUPPORTED), (dict(T=(1 << 26) - 3), UNSUPPORTED),
    (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE), (dict(logits=None), NULL), (dict(logits=ODD), ALIGN),
    (dict(ids=None), NULL), (dict(ids=ODD), ALIGN)])
def test_common(call, bad, status):
    assert call(**bad) == status
    assert moe.lib().moe_last_error()


@pytest.mark.parametrize("bad,status", [
    (dict(groups=0), SHAPE), (dict(groups=3), SHAPE), (dict(E=130, groups=65), UNSUPPORTED), (dict(kept=0), SHAPE),
    (dict(groups=4, kept=5), SHAPE), (dict(top=0), UNSUPPORTED), (dict(top=3), UNSUPPORTED),
    (dict(groups=8, kept=1, k=3), SHAPE), (dict(bias=ODD), ALIGN), (dict(w=None), NULL), (dict(w=ODD), ALIGN)])
def test_groups(bad, status):
    assert route(**bad) == status


def test_gradient_pointers():
    for bad in (dict(dw=None), dict(d=None)):
        assert backward(**bad) == NULL
    for bad in (dict(dw=ODD), dict(d=ODD)):
        assert backward(**bad) == ALIGN


def test_empty_calls_launch_nothing():
    assert route(T=0, logits=None, ids=None, w=None) == 0
    assert backward(T=0, logits=None, ids=None, dw=None, d=None) == 0


def test_binding():
    f32, i32 = torch.float32, torch.int32
    l, ids, w = Fake((4, 16), f32), Fake((4, 2), i32), Fake((4, 2), f32)
    grad = Fake((4, 16), f32)
    grad.requires_grad = True
    bad = [
        (lambda: moe.moe_route_topk(l, 2, scoring="tanh", out=(ids, w)), UNSUPPORTED),
        (lambda: moe.moe_route_topk(Fake((4, 16), torch.float64), 2, out=(ids, w)), UNSUPPORTED),
        (lambda: moe.moe_route_topk(Fake((4, 16), torch.uint8), 2, out=(ids, w)), UNSUPPORTED),
        (lambda: moe.moe_route_topk(Fake((4, 4, 16), f32), 2, out=(ids, w)), SHAPE),
        (lambda: moe.moe_route_topk(Fake((4, 16), f32, cuda=False, device="cpu"), 2, out=(ids, w)), SHAPE),
        (lambda: moe.moe_route_topk(Fake((4, 16), f32, dense=False), 2, out=(ids, w)), SHAPE),
        (lambda: moe.moe_route_topk(l, 2, bias=Fake((15,), f32), out=(ids, w)), SHAPE),
        (lambda: moe.moe_route_topk(l, 2, bias=Fake((16,)), out=(ids, w)), UNSUPPORTED),
        (lambda: moe.moe_route_topk(l, 2, bias=Fake((16,), f32, device="cuda:1"), out=(ids, w)), SHAPE),
        (lambda: moe.moe_route_topk(l, 3, out=(ids, w)), SHAPE),
        (lambda: moe.moe_route_topk(l, 2, out=(ids, Fake((4, 2)))), UNSUPPORTED),
        (lambda: moe.moe_route_topk(grad, 2, out=(ids, w)), UNSUPPORTED),
        (lambda: moe.moe_route_topk_backward(l, w, w, out=l), UNSUPPORTED),
        (lambda: moe.moe_route_topk_backward(l, ids, Fake((4, 3), f32), out=l), SHAPE),
        (lambda: moe.moe_route_topk_backward(l, ids, w, out=Fake((4, 16))), UNSUPPORTED),
        (lambda: moe.moe_route_topk_backward(grad, ids, w, out=l), UNSUPPORTED),
    ]
    for i, (call, status) in enumerate(bad):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == status, i
