"""The 4-bit FFN where one to five tokens have few and many routes per expert:
both ways to its second product on both sides of their rule.  Gates as in
test_gpu_w4.py."""

import numpy as np
import pytest
import torch

import mixture_experts_ffn_moe_amd as moe
from oracle import w4

from .test_gpu_w4 import check, activations, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,group,zeros", [("int4", 128, True), ("int4", 32, True), ("mx", 32, False)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 2), (1, 1, 3), (2, 3, 3), (2, 2, 3), (3, 4, 4), (4, 8, 4), (4, 6, 6), (4, 2, 8),
                                   (5, 3, 2)])
def test_ffn(T, E, k, fmt, group, zeros):
    rng = np.random.default_rng(T * E + k)
    K, I = 256, 640
    W1, D1 = weights(fmt, group, zeros, E, 2 * I, K, "bf16", rng)
    W2, D2 = weights(fmt, group, zeros, E, K, I, "bf16", rng)
    x, X = activations((T, K), "bf16", rng)
    # an expert twice in a token, and some routes elsewhere
    ids = rng.integers(0, E + 1, (T, k)).astype(np.int32)
    ids[:, 0] = 0
    w = rng.random((T, k)).astype(np.float32)
    w[ids == E] = np.nan
    out = torch.full((T, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((moe.moe_w4_workspace_size(T, K, 2 * I, k),), 0xFF, dtype=torch.uint8, device="cuda")
    got = moe.fused_moe_w4(fmt, X, *D1, *D2, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), group,
                           out=out, workspace=ws)
    ref, sigma = w4.ffn(fmt, W1, W2, group, x, ids, w, 1)
    check(got, ref, sigma, "bf16", "ffn")
    again = moe.fused_moe_w4(fmt, X, *D1, *D2, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), group)
    assert torch.equal(got, again)
