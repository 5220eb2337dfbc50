"""The general router with every number of slots a lane holds, with groups and
without: group counts that are no power of two leave lanes idle and the others with
more experts."""

import pytest
import torch

from .test_gpu_route_topk import check, logits_of

pytestmark = pytest.mark.gpu


def slots(E, G):
    """A lane's experts: lanes 2^lp a group, the most for which G groups fit."""
    lp = 6
    while G > 1 and (64 >> lp) < G:
        lp -= 1
    return -(-(E // G) // (1 << lp))


CASES = [(2, 1, 1), (4, 1, 256), (5, 1, 300), (8, 1, 500), (16, 1, 1023),
         (2, 16, 128), (2, 64, 128), (4, 8, 256), (4, 5, 155), (5, 64, 320), (5, 3, 240), (8, 33, 231), (8, 7, 448),
         (16, 2, 1024), (16, 33, 528), (16, 12, 768), (32, 33, 1023), (32, 17, 1020), (32, 9, 1017), (32, 5, 1020), (32, 3, 1023),
         (16, 63, 1008)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("NV,G,E", CASES)
def test_slots(NV, G, E, scoring):
    # the kernels hold 2, 4, 5, 8, 16 or 32
    assert next(n for n in (2, 4, 5, 8, 16, 32) if slots(E, G) <= n) == NV
    g = torch.Generator().manual_seed(E + G)
    bias = torch.randn(E, generator=g) * 0.3
    kept = max(1, G // 2)
    k = min(16, kept * (E // G))
    for elem, masked in (("f32", 0.0), ("f32", 0.7), ("bf16", 0.0), ("f16", 0.2)):
        l = logits_of(9, E, elem, E + G, masked)
        check(l, k, bias, elem, scoring=scoring, n_group=G, topk_group=kept, group_top=2, scale=2.5)
        check(l, 1, None, elem, scoring=scoring, n_group=G, topk_group=kept, group_top=1)
