"""The short way into the library (module _fast) takes plain calls only (CPU
only): anything else returns None, does nothing and raises nothing."""

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

from .test_rows_abi_cpu import Fake

F32, I32, F8 = torch.float32, torch.int32, torch.float8_e4m3fn


def fast():
    moe.lib()
    return moe._fast


def t(shape, dtype=F32):
    return torch.zeros(shape).to(dtype)


CALLS = [
    ("route_topk", lambda v: (v((4, 16)), None, v((4, 2), I32), v((4, 2)), 2, 0, 1, 1, 1, True, 1.0)),
    ("route_topk_backward", lambda v: (v((4, 16)), v((4, 2), I32), v((4, 2)), 0, True, 1.0, v((4, 16)))),
    ("fp8_quant", lambda v: (v((4, 32)), 0, True, False, None, v((4, 32), F8), v((4, 1)), None, None)),
    ("fp8_quant_weights", lambda v: (v((1, 16, 32)), 0, False, v((1, 16, 32), F8), v((1, 1, 1)), None, None)),
    ("fp8_linear", lambda v: (v((4, 32), F8), v((4, 1)), v((1, 16, 32), F8), v((1, 1, 1)), None, None, 0,
                              v((4, 16), torch.bfloat16))),
    ("fp8_linear_dw", lambda v: (v((16, 128), F8), v((16, 1)), v((32, 128), F8), v((32, 1)), 1, None, None, 0,
                                 v((1, 16, 32), torch.bfloat16))),
]


@pytest.mark.parametrize("name,args", CALLS, ids=[c[0] for c in CALLS])
def test_not_plain(name, args):
    f = getattr(fast(), name)
    assert f(*args(t)) is None  # no GPU tensors
    assert f(*args(Fake)) is None  # no tensors
    good = args(t)
    for i in range(len(good)):
        for odd in (None, "x", object(), 1 << 80, -1.5, [1], torch.zeros(0)):
            assert f(*good[:i], odd, *good[i + 1:]) is None
    assert f() is None and f(*good, None) is None


def test_lacking_library():
    with pytest.raises(Exception):
        fast().init("no handle", print)
    import ctypes
    with pytest.raises(RuntimeError):
        fast().init(ctypes.CDLL(None)._handle, print)
    moe._short_way(moe.lib())
