"""The operators on the rows of a plan where the rows are streamed past the
caches: more than 192 MiB of them.  Moved rows are compared bit by bit, sums
with fp64 on the device, under the bounds of test_gpu_rows.py: (n + 1) 2^-24 of
the terms' magnitudes for a sum of n products, and one rounding."""

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

from .test_gpu_rows import TINY, TYPES

pytestmark = pytest.mark.gpu

E, TOP_K, SHARED, BLOCK = 24, 6, 2, 128
STREAMED = 192 << 20


def make(elem, T, K, routed_to):
    """Inputs of T tokens, and of each row in use its token and its weight (0 rows of padding: token -1)."""
    g = torch.Generator(device="cuda").manual_seed(T + K)
    assert T * (TOP_K + SHARED) * K * TYPES[elem].itemsize > STREAMED
    ids = torch.rand(T, routed_to, device="cuda", generator=g).topk(TOP_K, dim=1).indices.int()
    plan, _, ntp = moe.moe_align_shared(ids, E, SHARED, BLOCK)
    row = moe.moe_route_rows(ids, E, plan, ntp, n_shared=SHARED)
    w = torch.rand(T, TOP_K, device="cuda", generator=g)
    n = int(ntp)
    r = plan[:n].long()
    routed = (r >= 0) & (r < T * TOP_K)
    token = torch.where(r < T * TOP_K, r // TOP_K, (r - T * TOP_K) // SHARED)
    token[r < 0] = -1
    weight = torch.where(routed, w.reshape(-1)[r.clamp(0, T * TOP_K - 1)], 1.0)
    return g, ids, plan, ntp, row, w, n, token, weight


def randn(g, shape, elem):
    return torch.randn(shape, device="cuda", generator=g).to(TYPES[elem])


def close(got, want, mag, terms, elem):
    u = torch.finfo(TYPES[elem]).eps / 2
    s = (terms + 1) * 2.0 ** -24 * mag
    assert bool((got.double() - want).abs().le(s + u * (want.abs() + s) + TINY[elem]).all())


def sums(rows, row, w, T, K):
    """The tokens' sums of 64-bit terms, and of their magnitudes, a few tokens at a time."""
    place = torch.cat((row[:T * TOP_K].reshape(T, TOP_K), row[T * TOP_K:].reshape(T, SHARED)), 1).long()
    wt = torch.cat((w, torch.ones(T, SHARED, device="cuda")), 1).double()
    for t in range(0, T, 512):
        p = place[t:t + 512]
        y = torch.where((p >= 0)[:, :, None], rows[p.clamp(min=0)].double() * wt[t:t + 512, :, None], 0.0)
        yield slice(t, t + 512), y.sum(1), y.abs().sum(1)


# a quarter of the routed experts elsewhere, and none
@pytest.mark.parametrize("elem,T,K,routed_to", [("bf16", 4096, 4096, 32), ("f16", 3333, 5128, 24), ("f32", 2048, 4096, 32)])
def test_streamed_rows(elem, T, K, routed_to):
    g, ids, plan, ntp, row, w, n, token, weight = make(elem, T, K, routed_to)
    cap = plan.numel()
    assert n < cap
    # into the rows: padding 0, rows past the plan left alone
    x = randn(g, (T, K), elem)
    rows = torch.full((cap, K), float("nan"), dtype=TYPES[elem], device="cuda")
    moe.moe_permute(x, row, plan, ntp, TOP_K, SHARED, out=rows)
    want = torch.where((token >= 0)[:, None], x[token.clamp(min=0)], 0.0)
    assert torch.equal(rows[:n], want) and bool(rows[n:].isnan().all())
    del want
    # and back, with the weights and without; what no route has is not read
    rows[:n] = randn(g, (n, K), elem)
    rows[:n][token < 0] = float("nan")
    got = moe.moe_unpermute(rows, row, w, TOP_K, SHARED)
    for t, ref, mag in sums(rows, row, w, T, K):
        close(got[t], ref, mag, TOP_K + SHARED, elem)
    got = moe.moe_permute_backward(rows, row, TOP_K, SHARED)
    for t, ref, mag in sums(rows, row, torch.ones_like(w), T, K):
        close(got[t], ref, mag, TOP_K + SHARED, elem)
    # the gradients of the weighted sum
    d_out = randn(g, (T, K), elem)
    buf = (torch.full((cap, K), float("nan"), dtype=TYPES[elem], device="cuda"),
           torch.full((T, TOP_K), float("nan"), device="cuda"))
    d_rows, d_w = moe.moe_unpermute_backward(d_out, rows, row, plan, ntp, w, TOP_K, SHARED, out=buf)
    assert bool(d_rows[n:].isnan().all())
    for p in range(0, n, 4096):
        t, wt = token[p:p + 4096], weight[p:p + 4096].double()
        ref = torch.where((t >= 0)[:, None], d_out[t.clamp(min=0)].double() * wt[:, None], 0.0)
        close(d_rows[p:p + 4096][:n - p], ref, ref.abs(), 1, elem)
    p = row[:T * TOP_K].reshape(T, TOP_K).long()
    for t in range(0, T, 512):
        y = rows[p[t:t + 512].clamp(min=0)].double() * d_out[t:t + 512, None].double()
        y = torch.where((p[t:t + 512] >= 0)[:, :, None], y, 0.0)
        err = (d_w[t:t + 512].double() - y.sum(-1)).abs()
        assert bool((err <= (K + 1) * 2.0 ** -24 * y.abs().sum(-1) + 2.0 ** -149).all())
    only, _ = moe.moe_unpermute_backward(d_out, None, row, plan, ntp, w, TOP_K, SHARED)
    assert torch.equal(only[:n], d_rows[:n])
