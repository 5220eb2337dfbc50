"""The calls on a plan's rows refuse inputs whose gradient autograd would lose
there (CPU only)."""

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

from .test_rows_abi_cpu import UNSUPPORTED, Fake


def fake(shape, dtype=torch.bfloat16, grad=False):
    t = Fake(shape, dtype)
    t.requires_grad = grad
    return t


def calls():
    i32, f32 = torch.int32, torch.float32
    row, plan, ntp, ids = (fake(s, i32) for s in ((8,), (64,), (1,), (4, 2)))
    x, rows, w = (lambda g: fake((4, 64), grad=g)), (lambda g: fake((64, 64), grad=g)), (lambda g: fake((4, 2), f32, g))
    to = fake((64, 64)), fake((4, 64)), fake((4, 2), f32), fake((4, 8), f32)
    return [
        lambda: moe.moe_permute(x(True), row, plan, ntp, 2, out=to[0]),
        lambda: moe.moe_permute_backward(rows(True), row, 2, out=to[1]),
        lambda: moe.moe_unpermute(rows(True), row, w(False), 2, out=to[1]),
        lambda: moe.moe_unpermute(rows(False), row, w(True), 2, out=to[1]),
        lambda: moe.moe_unpermute_backward(x(True), rows(False), row, plan, ntp, w(False), 2, out=(to[0], to[2])),
        lambda: moe.moe_unpermute_backward(x(False), rows(True), row, plan, ntp, None, 2, out=(to[0], to[2])),
        lambda: moe.moe_unpermute_backward(x(False), None, row, plan, ntp, w(True), 2, out=(to[0], None)),
        lambda: moe.moe_route_backward(ids, w(True), w(False), 8, out=to[3]),
        lambda: moe.moe_route_backward(ids, w(False), w(True), 8, out=to[3]),
    ]


@pytest.mark.parametrize("n", range(len(calls())))
def test_refused_with_gradients_enabled(n):
    with pytest.raises(moe.MoeError) as e:
        calls()[n]()
    assert e.value.status == UNSUPPORTED and "autograd" in str(e.value)


def test_taken_without():
    for t in (fake((2,), grad=True), fake((2,)), None):
        with torch.no_grad():
            moe._outside_autograd(t)
    moe._outside_autograd(fake((2,)), None)
