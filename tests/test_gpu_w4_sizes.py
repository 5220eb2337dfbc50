"""Sizes at which the products with 4-bit weights take another path: several
output tiles to a workgroup, a contraction walked in parts, more routes than
waves, contractions past a wave's LDS, and the FFN's two ways to its second
product.  Gates as in test_gpu_w4.py."""

import numpy as np
import pytest
import torch

import mixture_experts_ffn_moe_amd as moe
from oracle import w4

from .test_gpu_w4 import activations, check, parts, rounded, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,group,zeros", [("int4", 128, True), ("int4", 32, False), ("mx", 32, False)])
@pytest.mark.parametrize("elem,K,N", [("bf16", 256, 1050), ("f16", 128, 2090), ("bf16", 2048, 2080)])
def test_tiles_in_a_row(fmt, group, zeros, elem, K, N):
    """64 routes of 64 experts: two or four tiles a workgroup; exact."""
    rng = np.random.default_rng(N)
    E, T, k = 64, 32, 2
    W, D = weights(fmt, group, zeros, E, N, K, elem, rng, exact=True)
    x, X = activations((T, K), elem, rng, exact=True)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    ids[:6, 0] = 3                                   # more routes than a pass takes
    got = moe.moe_w4_matvec(fmt, X, *D, torch.from_numpy(ids).cuda(), group).double().cpu().numpy()
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        if e < 0:
            assert not got[t, j].any()
            continue
        d = w4.dequant(fmt, *[None if v is None else v[e] for v in W], group)
        assert np.array_equal(got[t, j], rounded(x[t] @ d.T, elem)), e


@pytest.mark.parametrize("fmt,group", [("int4", 128), ("int4", 64), ("mx", 32)])
@pytest.mark.parametrize("T,K,N", [(40, 1280, 22000), (16, 8192, 64), (9, 6144, 33), (3, 20480, 16), (1, 32768, 17)])
def test_contraction_in_parts(fmt, group, T, K, N):
    """A linear layer whose tokens do not fit the LDS at once; exact."""
    rng = np.random.default_rng(T)
    W, D = weights(fmt, group, False, 1, N, K, "bf16", rng, exact=True)
    x, X = activations((T, K), "bf16", rng, exact=True)
    x, X = np.clip(x, -2, 2), X.clamp(-2, 2)          # sums stay whole below 2^24
    got = moe.moe_w4_matvec(fmt, X, *D, None, group).double().cpu().numpy()
    d = w4.dequant(fmt, *[None if v is None else v[0] for v in W], group)
    assert np.array_equal(got, rounded(x @ d.T, "bf16"))


@pytest.mark.parametrize("fmt,group,zeros", [("int4", 128, True), ("int4", 64, False), ("int4", 32, True),
                                             ("mx", 32, False)])
@pytest.mark.parametrize("T,K,I,E,k", [(1, 128, 2176, 4, 3), (1, 256, 4480, 3, 2), (2, 128, 2048, 12, 11),
                                       (4, 256, 128, 20, 16), (5, 256, 2432, 6, 3), (1, 4096, 128, 9, 8)])
def test_ffn_paths(T, K, I, E, k, fmt, group, zeros):
    """Up to four tokens take a route per wave, more than that the grouped
    products; intermediates past a wave's LDS; more routes than waves."""
    rng = np.random.default_rng(I + k)
    W1, D1 = weights(fmt, group, zeros, E, 2 * I, K, "bf16", rng)
    W2, D2 = weights(fmt, group, zeros, E, K, I, "bf16", rng)
    x, X = activations((T, K), "bf16", rng)
    ids = np.stack([rng.permutation(E + 1)[:k] for _ in range(T)]).astype(np.int32) if k <= E else \
        rng.integers(0, E + 1, (T, k)).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    got = moe.fused_moe_w4(fmt, X, *D1, *D2, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), group)
    ref, sigma = w4.ffn(fmt, W1, W2, group, x, ids, w, parts("bf16"))
    check(got, ref, sigma, "bf16", "ffn")


def test_no_route_here():
    """Every route elsewhere: zeros, whatever the workspace held."""
    rng = np.random.default_rng(1)
    _, D1 = weights("int4", 64, True, 3, 128, 128, "bf16", rng)
    _, D2 = weights("int4", 64, True, 3, 128, 64, "bf16", rng)
    for T in (1, 7):
        x = torch.ones(T, 128, dtype=torch.bfloat16, device="cuda")
        ids = torch.full((T, 2), 3, dtype=torch.int32, device="cuda")
        ids[0, 0] = -5
        ws = torch.full((moe.moe_w4_workspace_size(T, 128, 128, 2),), 0xFF, dtype=torch.uint8, device="cuda")
        w = torch.full((T, 2), float("nan"), device="cuda")
        out = moe.fused_moe_w4("int4", x, *D1, *D2, ids, w, 64, workspace=ws)
        assert not bool(out.any()) and not bool(moe.moe_w4_matvec("int4", x, *D1, ids, 64).any())


@pytest.mark.parametrize("T", [4, 9])
def test_graph_of_both_paths(T):
    """Captured and replayed with other routing, beside eager work."""
    rng = np.random.default_rng(T)
    K, I, E, k = 256, 128, 6, 2
    _, D1 = weights("int4", 64, True, E, 2 * I, K, "f16", rng)
    _, D2 = weights("int4", 64, True, E, K, I, "f16", rng)
    x = torch.zeros(T, K, dtype=torch.float16, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    out = torch.empty_like(x)
    ws = torch.empty(moe.moe_w4_workspace_size(T, K, 2 * I, k), dtype=torch.uint8, device="cuda")

    def step(o, s):
        return moe.fused_moe_w4("int4", x, *D1, *D2, ids, w, 64, out=o, workspace=s)

    step(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, ws)
    for seed in (1, 2, 3):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(T, K, generator=g))
        ids.copy_(torch.randint(-1, E + 1, (T, k), generator=g))
        eager = step(torch.empty_like(x), torch.empty_like(ws)).clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), seed


def test_expert_past_4_gib():
    """The last of 520 experts, whose weights lie past 2^32 bytes; exact."""
    rng = np.random.default_rng(12)
    E, N, K = 520, 4096, 4096
    W, D = weights("int4", 128, True, 1, N, K, "bf16", rng, exact=True)
    w = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N, K // 128, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(E, N, K // 128, dtype=torch.uint8, device="cuda")
    w[-1], s[-1], z[-1] = D[0][0], D[1][0], D[2][0]
    x, X = activations((2, K), "bf16", rng, exact=True)
    ids = torch.full((2, 1), E - 1, dtype=torch.int32, device="cuda")
    got = moe.moe_w4_matvec("int4", X, w, s, z, ids, 128).double().cpu().numpy()
    d = w4.dequant("int4", *[v[0] for v in W], 128)
    assert np.array_equal(got[:, 0], rounded(x @ d.T, "bf16"))


@pytest.mark.parametrize("fmt,group", [("int4", 128), ("int4", 32), ("mx", 32)])
@pytest.mark.parametrize("elem,T,k,E,K,N", [
    ("bf16", 16, 1, 1, 4096, 72), ("bf16", 11, 1, 1, 4480, 64), ("f16", 8, 1, 1, 4096, 40),
    ("f16", 13, 1, 1, 1152, 4100), ("bf16", 16, 2, 8, 4096, 64), ("bf16", 150, 2, 8, 2048, 50),
    ("bf16", 2048, 2, 4, 4096, 32)])
def test_tokens_held_whole(fmt, group, elem, T, k, E, K, N):
    """Few output tiles of many tokens: the whole of K in a larger LDS; exact."""
    rng = np.random.default_rng(K + T)
    W, D = weights(fmt, group, fmt == "int4", E, N, K, elem, rng, exact=True)
    x, X = activations((T, K), elem, rng, exact=True)
    x, X = np.clip(x, -2, 2), X.clamp(-2, 2)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32) if E > 1 else None
    got = moe.moe_w4_matvec(fmt, X, *D, None if ids is None else torch.from_numpy(ids).cuda(), group)
    got = got.double().cpu().numpy().reshape(T, k, N)
    for e in range(E):
        t, j = np.nonzero(ids == e) if E > 1 else (np.arange(T), np.zeros(T, int))
        d = w4.dequant(fmt, *[None if v is None else v[e] for v in W], group)
        assert np.array_equal(got[t, j], rounded(x[t] @ d.T, elem)), e
    if E > 1:
        assert not got[ids < 0].any()


def test_first_call_captured():
    """A call whose kernels ask for more LDS than the default, in a graph with
    no eager call before it."""
    rng = np.random.default_rng(8)
    K, I, E, k = 256, 128, 9, 8
    _, D1 = weights("int4", 0, True, E, 2 * I, K, "f16", rng)
    _, D2 = weights("int4", 0, True, E, K, I, "f16", rng)
    _, DL = weights("int4", 0, True, 1, 64, 4096, "f16", rng)
    x = torch.randn(1, K, device="cuda").half()
    xl = torch.randn(8, 4096, device="cuda").half()
    ids = torch.arange(8, dtype=torch.int32, device="cuda").reshape(1, k)
    w = torch.full((1, k), 0.125, device="cuda")
    out, lin = torch.empty_like(x), torch.empty(8, 64, dtype=torch.float16, device="cuda")
    ws = torch.empty(moe.moe_w4_workspace_size(1, K, 2 * I, k), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.fused_moe_w4("int4", x, *D1, *D2, ids, w, 0, out=out, workspace=ws)
        moe.moe_w4_matvec("int4", xl, *DL, None, 0, out=lin)
    for seed in (1, 2, 3):
        x.copy_(torch.randn(1, K, generator=torch.Generator().manual_seed(seed)))
        xl.copy_(torch.randn(8, 4096, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe.fused_moe_w4("int4", x, *D1, *D2, ids, w, 0)), seed
        assert torch.equal(lin, moe.moe_w4_matvec("int4", xl, *DL, None, 0)), seed
