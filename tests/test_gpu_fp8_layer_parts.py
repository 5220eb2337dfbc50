"""The layer of experts of test_gpu_fp8_layer, step by step and part by part, small
and so large that the products run in 256 x 256 tiles.

Every quantized value is off by at most half a step of e4m3, 2^-4 of the value or
2^-10 of its scale (and one fp32 rounding of the scaled value); every 8-bit product
of a step is compared, per expert, with the fp64 product of the codes and scales that
it was given.  Activations and gradients have some values far above the rest, for which
the oracle's error model (like sizes, independent errors) is too small; the bound is
the instruction's own (test_gpu_mfma_groups): each product of eight loses less than
2^-13 of the eight's largest, which is at most the largest of x times the largest of w
there, and the fp32 additions, 17 for 128 and one between, each at most 2^-23 of the
products' absolute sum; and half a step of bf16.  Over a part these losses are a random
walk: in the 2-norm it is off by no more than half a step everywhere.

The whole against the layer in fp64 without quantization: per token and per expert,
so that one expert's lost gradient or one wrong row shows.  A product of two
quantized operands is off by 0.051 in the 2-norm (2^-4 / sqrt(3) for each), behind
the activation by at most three times that: output and second weights' gradient
sqrt(0.153^2 + 0.051^2) = 0.161, for parts of hundreds of elements below 0.25; first
weights' and input's gradient, the longest chains, below 0.49.  A part that is lost
or another's is off by 1 or more."""

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

from .test_gpu_fp8_layer import OPT, layer

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


def values(q, s):
    v = s.double() if s.dtype is torch.float32 else torch.exp2(s.double() - 127)
    return q.double() * v.repeat_interleave(128, 1)[:, :q.shape[1]], v.repeat_interleave(128, 1)[:, :q.shape[1]]


def blocks(q, s):
    v = s.double() if s.dtype is torch.float32 else torch.exp2(s.double() - 127)
    v = v.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * v, v


def close(got, x, w):
    y = x @ w.T.contiguous()
    X, W = (t.abs().reshape(len(t), -1, 8).amax(2) for t in (x, w))
    bound = 7 * 2.0 ** -13 * (X @ W.T.contiguous())
    bound += (18 * (x.shape[1] // 128 + 1) * 2.0 ** -23) * (x.abs() @ w.abs().T.contiguous())
    off = (got.detach().double() - y).abs()
    assert bool((off <= BF16 * y.abs() + 2.0 ** -134 + bound * (1 + BF16)).all())
    assert float(off.norm()) <= BF16 * float(y.norm())


def quantized(x, of):
    """x against (values, scales) of its codes."""
    v, s = of
    step = torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10) + x.abs() * 2.0 ** -23
    assert bool(((v - x).abs() <= step).all())


class Steps:
    """Records the calls a layer makes."""

    def __init__(self, monkeypatch):
        self.seen = []
        for name in ("moe_fp8_quant", "moe_fp8_quant_weights", "moe_fp8_linear", "moe_fp8_linear_dw"):
            monkeypatch.setattr(moe, name, self.recorder(name, getattr(moe, name)))

    def recorder(self, name, call):
        def f(*args, **more):
            result = call(*args, **more)
            self.seen.append((name, [v.detach().clone() if torch.is_tensor(v) else v for v in args], result))
            return result
        return f

    def check(self, experts, ntp, bm):
        n = int(ntp)
        of = experts.repeat_interleave(bm)[:n]
        for name, a, result in self.seen:
            if name == "moe_fp8_quant":
                x, (q, s, qt, st) = a[0][:n].double(), result
                quantized(x, [v[:n] for v in values(q, s)])
                cols, scales = values(qt, st)
                quantized(x, (cols[:, :n].T, scales[:, :n].T))
            elif name == "moe_fp8_quant_weights":
                q, s, qt, st = result
                for e in range(q.shape[0]):
                    quantized(a[0][e].double(), blocks(q[e], s[e]))
                    v, t = blocks(qt[e], st[e])
                    quantized(a[0][e].double(), (v.T, t.T))
            elif name == "moe_fp8_linear":
                x = values(a[0], a[1])[0]
                for e in range(a[2].shape[0]):
                    at = (of == e).nonzero()[:, 0]
                    close(result[at], x[at], blocks(a[2][e], a[3][e])[0])
            else:
                dy, x = values(a[0], a[1])[0], values(a[2], a[3])[0]
                for e in range(a[4]):
                    at = (of == e).nonzero()[:, 0]
                    close(result[e], dy[:, at], x[:, at])
        return [name for name, *_ in self.seen]


def off(got, want):
    """Relative 2-norms of the difference, row by row."""
    d, w = (got.detach().double() - want.detach()).flatten(1), want.detach().flatten(1)
    return (d.norm(dim=1) / w.norm(dim=1)).nan_to_num(nan=0.0, posinf=float("inf"))


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,K,I,E,k,bm", [(500, 272, 160, 8, 2, 128), (700, 528, 272, 6, 3, 256), (4300, 1024, 768, 8, 2, 128)])
def test_parts(T, K, I, E, k, bm, kind, monkeypatch):
    g = torch.Generator().manual_seed(T)
    x, gate = torch.randn(T, K, generator=g).bfloat16().float(), torch.randn(K, E, generator=g) / K ** 0.5
    w1, w2 = torch.randn(E, 2 * I, K, generator=g) / K ** 0.5, torch.randn(E, K, I, generator=g) / I ** 0.5
    v, bias = torch.randn(T, K, generator=g).cuda(), torch.randn(E, generator=g) * 0.1

    def act(y):
        return torch.nn.functional.silu(y[:, :I].float()).mul(y[:, I:].float()).to(y.dtype)

    steps = Steps(monkeypatch)
    X, G, W1, W2 = (t.cuda().requires_grad_() for t in (x, gate, w1, w2))
    out, ids = layer(X.bfloat16(), X @ G, bias.cuda(), W1, W2, k, bm, kind, act, OPT, True)
    (out.float() * v).sum().backward()
    monkeypatch.undo()
    plan, experts, ntp = moe.moe_align(ids, E, bm)
    names = steps.check(experts, ntp, bm)
    assert names.count("moe_fp8_linear") == 4 and names.count("moe_fp8_linear_dw") == 2 and names.count("moe_fp8_quant") == 4

    xd, gd, a, b = (t.double().cuda().requires_grad_() for t in (x, gate, w1, w2))
    sel = ids.long()
    s = torch.sigmoid(xd @ gd).gather(1, sel)
    w = s / s.sum(1, keepdim=True) * OPT["scale"]
    ref = torch.zeros_like(xd)
    for e in range(E):
        t, j = (sel == e).nonzero(as_tuple=True)
        h = xd[t] @ a[e].T.contiguous()
        h = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        ref = ref.index_add(0, t, w[t, j][:, None] * (h @ b[e].T.contiguous()))
    (ref * v.double()).sum().backward()
    assert float(off(out, ref).max()) < 0.25
    assert float(off(W2.grad, b.grad).max()) < 0.25
    assert float(off(W1.grad, a.grad).max()) < 0.49
    assert float(off(X.grad, xd.grad).max()) < 0.49
    assert float(off(G.grad[None], gd.grad[None]).max()) < 0.49
