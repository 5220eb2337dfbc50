"""The calls on a plan's rows as the steps of autograd functions: gradients of
a layer against fp64 autograd on the same routing, and against differences."""

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

pytestmark = pytest.mark.gpu


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row, plan, ntp, k):
        ctx.save_for_backward(row)
        ctx.k = k
        rows = torch.zeros(plan.numel(), x.shape[1], device=x.device)
        return moe.moe_permute(x, row, plan, ntp, k, out=rows)

    @staticmethod
    def backward(ctx, d_rows):
        return moe.moe_permute_backward(d_rows.contiguous(), *ctx.saved_tensors, ctx.k), None, None, None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w, row, plan, ntp, k):
        ctx.save_for_backward(rows, w, row, plan, ntp)
        ctx.k = k
        return moe.moe_unpermute(rows, row, w, k)

    @staticmethod
    def backward(ctx, d_out):
        rows, w, row, plan, ntp = ctx.saved_tensors
        buf = torch.zeros_like(rows), None
        return (*moe.moe_unpermute_backward(d_out.contiguous(), rows, row, plan, ntp, w, ctx.k, out=buf),
                None, None, None, None)


class Weights(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, w):
        ctx.save_for_backward(ids, w)
        ctx.E = logits.shape[1]
        return w.clone()

    @staticmethod
    def backward(ctx, d_w):
        return moe.moe_route_backward(*ctx.saved_tensors, d_w.contiguous(), ctx.E), None, None


@pytest.mark.parametrize("T,K,E,k", [(37, 64, 5, 2), (1, 40, 3, 3), (66, 9, 4, 1)])
def test_layer_gradients(T, K, E, k):
    g = torch.Generator().manual_seed(T)
    x, gate, v = torch.randn(T, K, generator=g), torch.randn(K, E, generator=g) / 8, torch.randn(T, K, generator=g)
    scale = torch.randn(E, K, generator=g)
    X, G = x.cuda().requires_grad_(), gate.cuda().requires_grad_()
    logits = X @ G
    ids, w0, plan, experts, ntp = moe.moe_route_align(logits.detach(), k, 16)
    row = moe.moe_route_rows(ids, E, plan, ntp)
    w = Weights.apply(logits, ids, w0)
    rows = Gather.apply(X, row, plan, ntp, k)
    e_of = experts.clamp(min=0).long().repeat_interleave(16)[:plan.numel()]
    y = torch.tanh(rows * scale.cuda()[e_of])
    out = Combine.apply(y, w, row, plan, ntp, k)
    (out * v.cuda()).sum().backward()

    sel = ids.cpu().long()

    def layer(xd, gd):
        wd = torch.softmax((xd @ gd).gather(1, sel), 1)
        return sum(wd[:, j:j + 1] * torch.tanh(xd * scale.double()[sel[:, j]]) for j in range(k))

    xd, gd = x.double().requires_grad_(), gate.double().requires_grad_()
    loss = (layer(xd, gd) * v.double()).sum()
    loss.backward()
    # fp32 steps: sums of T, K or k terms of order one, and tanh's own few steps
    # (the largest magnitudes here are below 64)
    tol = (T + K + 16) * 2.0 ** -24 * 64
    assert float((out.detach().cpu().double() - layer(xd, gd).detach()).abs().max()) < tol
    assert float((X.grad.cpu().double() - xd.grad).abs().max()) < tol
    assert float((G.grad.cpu().double() - gd.grad).abs().max()) < tol * T
    # and by differences along a direction, in fp64: step^2 of a third derivative
    # and 2^-53 / step of the loss
    d, step = torch.randn(T, K, generator=g).double(), 1e-5
    with torch.no_grad():
        up, down = (layer(xd + s * d, gd) for s in (step, -step))
        num = float(((up - down) * v.double()).sum() / (2 * step))
    got = float((X.grad.cpu().double() * d).sum())
    assert abs(got - num) < tol * T * K + 1e-5


def test_refused_outside():
    x = torch.ones(2, 8, device="cuda", requires_grad=True)
    ids = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    plan, _, ntp = moe.moe_align(ids, 1, 16)
    row = moe.moe_route_rows(ids, 1, plan, ntp)
    with pytest.raises(moe.MoeError):
        moe.moe_permute(x, row, plan, ntp, 1)
    with torch.no_grad():
        assert torch.equal(moe.moe_permute(x, row, plan, ntp, 1)[:2], x.detach())
