"""What the products with 4-bit weights keep of their sums and of the FFN's
intermediate: results that are small differences of large terms.

Where nothing else is said every value is a whole multiple of a power of two, and
every sum that fp32 and the documented operands need stays below 2^24 of that
power, so each result is exact."""

import numpy as np
import pytest
import torch

import mixture_experts_ffn_moe_amd as moe
from oracle import w4

from .test_gpu_w4 import check
from .test_oracle_w4_types import cancelling

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
INT4 = [(32, True), (32, False), (64, True), (128, False), (128, True), (0, False)]


def codes(shape, fill, at):
    """Packed codes: ``fill`` everywhere but at {index: code}."""
    q = torch.full(shape, fill, dtype=torch.uint8)
    for i, c in at.items():
        q[i] = c
    return (q[..., 0::2] | q[..., 1::2] << 4).contiguous().cuda()


def int4(shape, group, zeros, at, elem):
    """Weights of 0 but at {index: whole value}, scale 1."""
    E, N, K = shape
    n = K // group if group else 1
    w = codes(shape, 8, {i: 8 + v for i, v in at.items()})
    z = torch.full((E, N, n), 8, dtype=torch.uint8, device="cuda") if zeros else None
    return [w, torch.ones(E, N, n, dtype=TYPES[elem], device="cuda"), z]


@pytest.mark.parametrize("elem", list(TYPES))
@pytest.mark.parametrize("group,zeros", INT4)
@pytest.mark.parametrize("T", [1, 3, 16, 20])
def test_int4_sum_cancels(T, group, zeros, elem):
    """1 - 1 + 2^-17: with codes held as 16 + q the sums reach 48, 2^23 times
    2^-18 (an offset of 128 takes them to 272, whose fp32 step is 2^-15)."""
    K, N = 512, 24
    # the three terms in one group: of one instruction, and of several
    places = {n: (32 * (n % 16), 32 * (n % 16) + 1 + n, 32 * (n % 16) + 31) for n in range(N)}
    shift = torch.arange(T) % 5
    out = []
    for n, (a, b, c) in places.items():
        W = int4((1, 8, K), group, zeros, {(0, n % 8, a): 1, (0, n % 8, b): -1, (0, n % 8, c): 1}, elem)
        x = torch.zeros(T, K)
        x[:, a] = x[:, b] = 2.0 ** shift
        x[:, c] = 2.0 ** (shift - 17)
        out.append(moe.moe_w4_matvec("int4", x.to(TYPES[elem]).cuda(), *W, None, group)[:, n % 8])
    want = (2.0 ** (shift - 17)).to(TYPES[elem])
    for n, y in enumerate(out):
        assert torch.equal(y.cpu(), want), (n, y.tolist())


def e2m1(shape, at, scales):
    """Weights of 0 but at {index: sign}, each 1 times the scale of its row."""
    E, N, K = shape
    w = codes(shape, 0, {i: 2 if v > 0 else 10 for i, v in at.items()})
    s = torch.full((E, N, K // 32), 127, dtype=torch.uint8)
    for row, e in scales.items():
        s[:, row] = 127 + e
    return [w, s.cuda(), None]


def cancelling_ffn(fmt, group, zeros, K, I, a, b, elem):
    """W1 and W2 of one expert: h[a] and h[b] are 32 x0 times x0 + x1 + x2 and x0 + x1 (gate 32 x0, past which
    silu is the identity in fp32), every other h is 0, and output n is h[a] - h[b] or, where n is odd, the reverse."""
    gate = {(0, a, 0): 1, (0, b, 0): 1}
    up = {(0, I + a, 0): 1, (0, I + a, 1): 1, (0, I + a, 2): 1, (0, I + b, 0): 1, (0, I + b, 1): 1}
    down = {}
    for n in range(K):
        down[(0, n, a)], down[(0, n, b)] = (1, -1) if n % 2 == 0 else (-1, 1)
    if fmt == "mx":
        return e2m1((1, 2 * I, K), {**gate, **up}, {a: 5, b: 5}), e2m1((1, K, I), down, {})
    W1 = int4((1, 2 * I, K), group, zeros, {**gate, **up}, elem)
    W1[1][:, [a, b]] = 32
    return W1, int4((1, K, I), group, zeros, down, elem)


@pytest.mark.parametrize("elem", list(TYPES))
@pytest.mark.parametrize("fmt,group,zeros", [("mx", 32, False), ("int4", 32, True), ("int4", 64, False),
                                             ("int4", 128, True)])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 9, 20])
def test_intermediate_keeps_fp32(T, fmt, group, zeros, elem):
    """h[a] - h[b] = 32 (1 + 2^-9 + 2^-17) - 32 (1 + 2^-9): bf16 parts of 8 bits, rounded, need three of them.  a and
    b lie in two scale groups, where 25 h and 24 h (codes held as 16 + q) take 23 bits of 2^-13."""
    K, I = 128, 512
    W1, W2 = cancelling_ffn(fmt, group, zeros, K, I, 37, 300, elem)
    shift = (torch.arange(T) % 4).double()
    x = torch.zeros(T, K)
    x[:, 0], x[:, 1], x[:, 2] = 2.0 ** shift, 2.0 ** (shift - 9), 2.0 ** (shift - 17)
    ids = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.5]], device="cuda").repeat(T, 1)
    got = moe.fused_moe_w4(fmt, x.to(TYPES[elem]).cuda(), *W1, *W2, ids, w, group).cpu()
    want = 32 * 4.0 ** shift * 2.0 ** -17
    sign = torch.tensor([1.0, -1.0]).repeat(K // 2)
    assert torch.equal(got.double(), want[:, None] * sign[None].double()), got[:, :2].tolist()


@pytest.mark.parametrize("T", [1, 6])
def test_intermediate_near_the_largest(T):
    """h just below 2^128, which rounds to infinity in bf16, and h past it."""
    K, I = 128, 128
    W1 = e2m1((1, 2 * I, K), {(0, 3, 0): 1, (0, I + 3, 1): 1, (0, I + 3, 2): 1, (0, 5, 0): 1, (0, I + 5, 3): 1}, {})
    W2 = e2m1((1, K, I), {(0, 0, 3): 1, (0, 1, 5): -1}, {0: -20, 1: -20})
    x = torch.zeros(T, K)
    x[:, 0], x[:, 1], x[:, 2], x[:, 3] = 2.0 ** 64, 2.0 ** 63 * 255 / 128, 2.0 ** 55, 2.0 ** 66
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(T, 1, device="cuda")
    # h[5] is infinite: the infinity, and NaN where a weight of 0 meets it (output 0 too: 0 times infinity)
    got = moe.fused_moe_w4("mx", x.bfloat16().cuda(), *W1, *W2, ids, w, 32).cpu().float()
    assert bool((got[:, 1] == float("-inf")).all())
    assert bool(got[:, 0].isnan().all()) and bool(got[:, 2:].isnan().all())
    x[:, 3] = 0                                         # h[5] is 0
    got = moe.fused_moe_w4("mx", x.bfloat16().cuda(), *W1, *W2, ids, w, 32).cpu().float()
    assert bool((got[:, 0] == 2.0 ** 108).all())        # 511 / 256 2^107, rounded to bf16
    assert not bool(got[:, 1:].any())


@pytest.mark.parametrize("group,zeros", [(128, False), (128, True), (64, True), (32, True)])
@pytest.mark.parametrize("T", [1, 5, 19])
def test_fp16_sums_of_large_terms(T, group, zeros):
    """Within six deviations of the error model for codes held as q - 8."""
    rng = np.random.default_rng(T + group)
    w, s, z, x = cancelling(group, zeros, 48, 512, T, rng)
    dev = [torch.from_numpy(w)[None].cuda(), torch.from_numpy(s).half()[None].cuda(),
           None if z is None else torch.from_numpy(z)[None].cuda()]
    got = moe.moe_w4_matvec("int4", torch.from_numpy(x).half().cuda(), *dev, None, group)
    ref = [w4.product("int4", w, s, z, group, v, *w4.operands("int4", "f16")) for v in x]
    check(got, np.stack([y for y, _ in ref]), np.stack([d for _, d in ref]), "f16", "large terms")
