"""The general router and the 8-bit operators run together as a layer of
experts, forward and backward: route, plan, permute, quantize, product,
activation, quantize, product, unpermute, and every gradient.

Exact: values whose quantization is exact (few significant bits, one weight a
row), so that outputs and gradients are those of the layer in fp64, rounded
once.  Real: an ordinary layer against fp64 autograd without quantization.  An
e4m3 rounding is off by at most 2^-4 of a value, 2^-4 / sqrt(3) = 0.036 in the
mean square over evenly spread fractions; a product of two such operands by
sqrt(2) times that, 0.051, in the 2-norm.  The longest chain of a result here is
three products with the activation's derivative between (a factor below 3 on the
error): sqrt((3 (3 * 0.051 + 0.051) + 0.051)^2) < 0.67 if all errors agreed in
sign; they are independent, so that sqrt((9 * 0.051)^2 + (3 * 0.051)^2 + 0.051^2) <
0.49 bounds the 2-norm, and a single wrong index or a lost scale is off by 1 or
more."""

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

pytestmark = pytest.mark.gpu


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, k, opt):
        ids, w = moe.moe_route_topk(logits, k, bias, **opt)
        ctx.save_for_backward(logits, ids)
        ctx.opt = {n: opt[n] for n in ("scoring", "renormalize", "scale")}
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    def backward(ctx, _, d_w):
        return moe.moe_route_topk_backward(*ctx.saved_tensors, d_w.contiguous(), **ctx.opt), None, None, None


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row, plan, ntp, k):
        ctx.save_for_backward(row)
        ctx.k = k
        return moe.moe_permute(x, row, plan, ntp, k, out=torch.zeros(plan.numel(), x.shape[1], dtype=x.dtype, device="cuda"))

    @staticmethod
    def backward(ctx, d):
        return moe.moe_permute_backward(d.contiguous(), *ctx.saved_tensors, ctx.k), None, None, None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w, row, plan, ntp, k):
        ctx.save_for_backward(rows, w, row, plan, ntp)
        ctx.k = k
        return moe.moe_unpermute(rows, row, w, k)

    @staticmethod
    def backward(ctx, d):
        rows, w, row, plan, ntp = ctx.saved_tensors
        out = torch.zeros_like(rows), None
        d_rows, d_w = moe.moe_unpermute_backward(d.contiguous(), rows, row, plan, ntp, w, ctx.k, out=out)
        return d_rows, None if w is None else d_w, None, None, None, None


class Linear(torch.autograd.Function):
    """rows (bf16) times an expert's weights (fp32 parameters), all three products in 8 bits."""

    @staticmethod
    def forward(ctx, rows, w, experts, ntp, bm, kind):
        q, s, qt, st = moe.moe_fp8_quant(rows, kind, columns=True, num_tokens_post_padded=ntp)
        wq, ws, wt, wts = moe.moe_fp8_quant_weights(w, kind, transposed=True)
        ctx.save_for_backward(qt, st, wt, wts, experts, ntp)
        ctx.bm, ctx.kind, ctx.E = bm, kind, w.shape[0]
        out = torch.zeros(rows.shape[0], w.shape[1], dtype=rows.dtype, device="cuda")
        return moe.moe_fp8_linear(q, s, wq, ws, experts, ntp, bm, out=out)

    @staticmethod
    def backward(ctx, d):
        qt, st, wt, wts, experts, ntp = ctx.saved_tensors
        q, s, dt, dts = moe.moe_fp8_quant(d.contiguous(), ctx.kind, columns=True, num_tokens_post_padded=ntp)
        d_rows = torch.zeros(d.shape[0], wt.shape[1], dtype=d.dtype, device="cuda")
        moe.moe_fp8_linear(q, s, wt, wts, experts, ntp, ctx.bm, out=d_rows)
        d_w = moe.moe_fp8_linear_dw(dt, dts, qt, st, ctx.E, experts, ntp, ctx.bm)
        return d_rows, d_w.float(), None, None, None, None


def layer(x, logits, bias, w1, w2, k, bm, kind, act, opt, weighted):
    ids, w = Route.apply(logits, bias, k, opt)
    plan, experts, ntp = moe.moe_align(ids, w1.shape[0], bm)
    row = moe.moe_route_rows(ids, w1.shape[0], plan, ntp)
    rows = Gather.apply(x, row, plan, ntp, k)
    y = act(Linear.apply(rows, w1, experts, ntp, bm, kind))
    y = Linear.apply(y, w2, experts, ntp, bm, kind)
    return Combine.apply(y, w if weighted else None, row, plan, ntp, k), ids


OPT = dict(scoring="sigmoid", n_group=2, topk_group=1, group_top=2, renormalize=True, scale=1.5)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,K,N,E,bm", [(200, 256, 144, 6, 128), (300, 144, 272, 4, 256), (1, 32, 16, 4, 128)])
def test_exact(T, K, N, E, bm, kind):
    k = 2
    g = torch.Generator().manual_seed(T)

    def picks(n, m):  # one weight of +-1 or 2 a row, and one a column at most
        w = torch.zeros(E, n, m)
        for e in range(E):
            r = torch.arange(min(n, m))
            w[e, torch.randperm(n, generator=g)[r], torch.randperm(m, generator=g)[r]] = \
                torch.tensor([1.0, -1.0, 2.0])[torch.randint(0, 3, r.shape, generator=g)]
        return w

    x = torch.randint(-2, 3, (T, K), generator=g).float()
    v = torch.randint(-1, 2, (T, K), generator=g).float()
    logits, bias = torch.randn(T, E, generator=g), torch.randn(E, generator=g) * 0.1
    w1, w2 = picks(N, K), picks(K, N)
    X = x.bfloat16().cuda().requires_grad_()
    W1, W2 = w1.cuda().requires_grad_(), w2.cuda().requires_grad_()
    act = lambda y: torch.where(y > 0, 2 * y, y)  # noqa: E731
    out, ids = layer(X, logits.cuda(), bias.cuda(), W1, W2, k, bm, kind, act, OPT, False)
    (out.float() * v.cuda()).sum().backward()

    xd, a, b = x.double().requires_grad_(), w1.double().requires_grad_(), w2.double().requires_grad_()
    sel = ids.cpu().long()
    ref = sum(torch.einsum("tn,tkn->tk", act(torch.einsum("tk,tnk->tn", xd, a[sel[:, j]])), b[sel[:, j]]) for j in range(k))
    (ref * v.double()).sum().backward()

    def same(got, want):
        assert torch.equal(got.detach().cpu().double(), want.detach().bfloat16().double())

    same(out, ref)
    same(X.grad, xd.grad)
    same(W1.grad, a.grad)
    same(W2.grad, b.grad)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_real(kind):
    T, K, I, E, k, bm = 500, 272, 160, 8, 2, 128
    g = torch.Generator().manual_seed(1)
    x, gate = torch.randn(T, K, generator=g), torch.randn(K, E, generator=g) / K ** 0.5
    w1, w2 = torch.randn(E, 2 * I, K, generator=g) / K ** 0.5, torch.randn(E, K, I, generator=g) / I ** 0.5
    v, bias = torch.randn(T, K, generator=g), torch.randn(E, generator=g) * 0.1

    def act(y):
        return torch.nn.functional.silu(y[:, :I].float()).mul(y[:, I:].float()).to(y.dtype)

    X, G = x.cuda().requires_grad_(), gate.cuda().requires_grad_()
    W1, W2 = w1.cuda().requires_grad_(), w2.cuda().requires_grad_()
    out, ids = layer(X.bfloat16(), X @ G, bias.cuda(), W1, W2, k, bm, kind, act, OPT, True)
    (out.float() * v.cuda()).sum().backward()

    xd, gd, a, b = (t.double().requires_grad_() for t in (x, gate, w1, w2))
    sel = ids.cpu().long()
    s = torch.sigmoid(xd @ gd).gather(1, sel)
    w = s / s.sum(1, keepdim=True) * OPT["scale"]
    ref = 0
    for j in range(k):
        h = torch.einsum("tk,tnk->tn", xd, a[sel[:, j]])
        h = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        ref = ref + w[:, j:j + 1] * torch.einsum("tn,tkn->tk", h, b[sel[:, j]])
    (ref * v.double()).sum().backward()
    for got, want in ((out, ref), (X.grad, xd.grad), (G.grad, gd.grad), (W1.grad, a.grad), (W2.grad, b.grad)):
        off = torch.linalg.norm(got.detach().cpu().double() - want.detach()) / torch.linalg.norm(want.detach())
        assert float(off) < 0.49


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_decode_step_replays(kind):
    """A step of few tokens as a server captures it: route, plan, permute as bytes, product."""
    T, K, N, E, k, bm = 9, 256, 200, 16, 4, 16
    g = torch.Generator().manual_seed(4)
    w = torch.randn(E, N, K, generator=g).cuda() / 16
    wq, ws, _, _ = moe.moe_fp8_quant_weights(w, kind)
    x, logits = torch.randn(T, K, generator=g).bfloat16().cuda(), torch.randn(T, E, generator=g).cuda()
    rows, blocks = moe.moe_align_capacity(T, k, E, bm)
    t = dict(dtype=torch.int32, device="cuda")
    ids, wt = torch.empty(T, k, **t), torch.empty(T, k, device="cuda")
    plan, experts, ntp, row = torch.empty(rows, **t), torch.empty(blocks, **t), torch.empty(1, **t), torch.empty(T * k, **t)
    scale = torch.float32 if kind == "f32" else torch.uint8
    q = torch.empty(T, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, 2, dtype=scale, device="cuda"), None, None
    pq = torch.zeros(rows, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(rows, 2, dtype=scale, device="cuda")
    y, out = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")

    def step():
        moe.moe_route_topk(logits, k, scoring="sigmoid", out=(ids, wt))
        moe.moe_align(ids, E, bm, out=(plan, experts, ntp))
        moe.moe_route_rows(ids, E, plan, ntp, out=row)
        moe.moe_fp8_quant(x, kind, out=q)
        moe.moe_permute(q[0], row, plan, ntp, k, out=pq[0])
        moe.moe_permute(q[1], row, plan, ntp, k, out=pq[1])
        moe.moe_fp8_linear(*pq, wq, ws, experts, ntp, bm, out=y)
        return moe.moe_unpermute(y, row, wt, k, out=out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6, 7):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(T, K, generator=g))
        logits.copy_(torch.randn(T, E, generator=g) * 3)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        assert torch.equal(got, out)
        p = torch.sigmoid(logits.double().cpu())
        ww, sel = p.topk(k, dim=1)
        ref = (torch.einsum("tk,tjnk->tjn", x.double().cpu(), w.double().cpu()[sel]) * (ww / ww.sum(1, keepdim=True))[..., None]).sum(1)
        assert torch.linalg.norm(got.double().cpu() - ref) < 0.08 * torch.linalg.norm(ref)  # one product: 0.051
