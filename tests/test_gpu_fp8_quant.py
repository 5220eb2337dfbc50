"""GPU parity of the 8-bit quantizers: codes and scales are those of the oracle
(oracle/fp8.py), bit for bit."""

import numpy as np
import pytest
import torch

import mixture_experts_ffn_moe_amd as moe
from oracle import fp8

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
KINDS = ("f32", "e8m0")
MARK = 0x55


def values(shape, elem, seed, wide=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if wide:
        x *= torch.exp(2 * torch.randn(shape[:-1] + (1,), generator=g))
    return x.to(TYPES[elem])


def buffers(M, K, kind, rows=True, columns=True):
    t = torch.float32 if kind == "f32" else torch.uint8
    G = -(-M // 128)
    made = [((M, K), torch.uint8), ((M, -(-K // 128)), t), ((K, 128 * G), torch.uint8), ((K, G), t)]
    out = [torch.full(s, MARK, dtype=d, device="cuda") for s, d in made]
    out[0], out[2] = out[0].view(torch.float8_e4m3fn), out[2].view(torch.float8_e4m3fn)
    return tuple(o if (rows if i < 2 else columns) else None for i, o in enumerate(out))


def same(q, s, ref):
    return np.array_equal(q.view(torch.uint8).cpu().numpy(), ref[0]) and np.array_equal(s.cpu().numpy(), ref[1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (17, 256), (127, 400), (128, 128), (129, 48), (200, 1040),
                                 (5, 4112), (300, 176)])
def test_forms(M, K, kind):
    for elem in TYPES:
        x = values((M, K), elem, M + K)
        f = x.float().numpy()
        rows, cols = fp8.quant_rows(f, kind), fp8.quant_columns(f, kind)
        for r, c in ((True, False), (False, True), (True, True)):
            q, s, qt, st = moe.moe_fp8_quant(x.cuda(), kind, rows=r, columns=c, out=buffers(M, K, kind, r, c))
            assert not r or same(q, s, rows), (elem, r, c)
            assert not c or same(qt, st, cols), (elem, r, c)
            assert (q is None) == (not r) and (qt is None) == (not c)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (3, 144, 272), (2, 16, 400), (1, 300, 160)])
def test_weights(E, N, K, kind):
    for elem in TYPES:
        w = values((E, N, K), elem, N + K, wide=False)
        for turned in (False, True) if N % 16 == 0 else (False,):
            q, s, qt, st = moe.moe_fp8_quant_weights(w.cuda(), kind, turned)
            for e in range(E):
                ref = fp8.quant_blocks(w[e].float().numpy(), kind)
                assert same(q[e], s[e], ref)
                assert not turned or same(qt[e], st[e], (ref[0].T, ref[1].T))
            assert (qt is None) == (not turned)


@pytest.mark.parametrize("kind", KINDS)
def test_extremes(kind):
    # zeros, the floor, tiny and huge groups, the border of a power of two
    x = torch.zeros(8, 128)
    x[1, 3] = 1e-30
    x[2, :2] = torch.tensor([1e-12, -3e-14])
    x[3, 0] = 3.3e38
    x[4, :3] = torch.tensor([448.0, 447.0, -1e-3])
    x[5, 0] = float(np.nextafter(np.float32(448), np.float32(1000)))
    x[6] = torch.linspace(-1, 1, 128)
    x[7, 0] = 1e-38
    f = x.numpy()
    q, s, qt, st = moe.moe_fp8_quant(x.cuda(), kind, columns=True)
    assert same(q, s, fp8.quant_rows(f, kind)) and same(qt, st, fp8.quant_columns(f, kind))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_not_finite(kind, bad):
    for elem in ("bf16", "f16", "f32"):
        x = values((130, 256), elem, 3)
        x[5, 200] = bad
        q, s, qt, st = moe.moe_fp8_quant(x.cuda(), kind, columns=True)
        clean = values((130, 256), elem, 3)
        c = moe.moe_fp8_quant(clean.cuda(), kind, columns=True)

        def what(q, s):
            v = s.double() if kind == "f32" else torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127))
            return q.float().double() * v.repeat_interleave(128, 1)

        rows, cols = what(q, s), what(qt, st)
        assert rows[5, 128:].isnan().all() and cols[200, :128].isnan().all()
        rows[5, 128:] = what(c[0], c[1])[5, 128:]
        cols[200, :128] = what(c[2], c[3])[200, :128]
        assert torch.equal(rows, what(c[0], c[1])) and torch.equal(cols, what(c[2], c[3]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,ntp", [(300, 0), (300, 1), (300, 128), (300, 200), (300, 300), (300, 999), (300, -4)])
def test_rows_in_use(M, ntp, kind):
    K, n = 144, max(0, min(ntp, M))
    x = values((M, K), "bf16", M)
    x[n:] = float("nan")  # neither read nor written
    count = torch.tensor([ntp], dtype=torch.int32, device="cuda")
    for c in (False, True):
        out = buffers(M, K, kind, True, c)
        q, s, qt, st = moe.moe_fp8_quant(x.cuda(), kind, columns=c, num_tokens_post_padded=count, out=out)
        mark = buffers(M, K, kind)
        f = x[:n].float().numpy()
        if n:
            assert same(q[:n], s[:n], fp8.quant_rows(f, kind))
        assert torch.equal(q[n:].view(torch.uint8), mark[0][n:].view(torch.uint8)) and torch.equal(s[n:], mark[1][n:])
        if c:
            g = -(-n // 128)
            if n:
                assert same(qt[:, :128 * g], st[:, :g], fp8.quant_columns(f, kind))
            assert torch.equal(qt[:, 128 * g:].view(torch.uint8), mark[2][:, 128 * g:].view(torch.uint8))
            assert torch.equal(st[:, g:], mark[3][:, g:])


def test_empty_and_larger():
    q, s, qt, st = moe.moe_fp8_quant(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), columns=True)
    assert q.shape == (0, 64) and qt.shape == (64, 0)
    x = values((1031, 2064), "bf16", 8)
    q, s, qt, st = moe.moe_fp8_quant(x.cuda(), "e8m0", columns=True)
    f = x.float().numpy()
    at = [0, 127, 128, 640, 1030]
    assert same(q[at], s[at], fp8.quant_rows(f[at], "e8m0"))
    assert same(qt[::333], st[::333], fp8.quant_columns(np.ascontiguousarray(f[:, ::333]), "e8m0"))


def test_captured_replays():
    x, w = values((100, 256), "bf16", 1).cuda(), values((2, 64, 256), "f32", 2).cuda()
    out, wout = buffers(100, 256, "f32"), moe.moe_fp8_quant_weights(w, transposed=True)

    def call():
        moe.moe_fp8_quant(x, columns=True, out=out)
        moe.moe_fp8_quant_weights(w, transposed=True, out=wout)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (3, 4, 5):
        x.copy_(values((100, 256), "bf16", seed))
        w.copy_(values((2, 64, 256), "f32", seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.view(torch.uint8).clone() for v in (*out, *wout)]
        call()
        assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(got, (*out, *wout)))
