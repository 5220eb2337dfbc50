"""What the products with 4-bit weights keep of their sums and of the FFN's
intermediate: results that are small differences of large terms.

Every value below is a whole multiple of a power of two, and every sum that
fp32 and the documented operands need stays below 2^24 of that power, so each
result is exact."""

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

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
