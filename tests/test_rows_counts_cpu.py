"""Expert counts past the C ABI's 32 bits are refused, not cut off (CPU only)."""

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

from .test_rows_abi_cpu import SHAPE
from .test_rows_autograd_cpu import fake


@pytest.mark.parametrize("E", [0, -1, 1 << 31, (1 << 32) + 8])
def test_expert_counts(E):
    i32, f32 = torch.int32, torch.float32
    ids, plan, ntp, w = fake((4, 2), i32), fake((64,), i32), fake((1,), i32), fake((4, 2), f32)
    for call in (lambda: moe.moe_route_rows(ids, E, plan, ntp, out=fake((8,), i32)),
                 lambda: moe.moe_route_backward(ids, w, w, E, out=fake((4, max(E, 0)), f32))):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == SHAPE
