"""Without module _fast, or with one that was built for another torch, the library
loads and every call goes the ordinary way (CPU only)."""

import os
import subprocess
import sys

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, I32, F8, BF16 = torch.float32, torch.int32, torch.float8_e4m3fn, torch.bfloat16


def t(shape, dtype=F32):
    return torch.zeros(shape).to(dtype)


CALLS = {
    "moe_route_topk": lambda: moe.moe_route_topk(t((4, 16)), 2, out=(t((4, 2), I32), t((4, 2)))),
    "moe_route_topk_backward": lambda: moe.moe_route_topk_backward(t((4, 16)), t((4, 2), I32), t((4, 2)), out=t((4, 16))),
    "moe_fp8_quant": lambda: moe.moe_fp8_quant(t((4, 32)), out=(t((4, 32), F8), t((4, 1)), None, None)),
    "moe_fp8_quant_weights": lambda: moe.moe_fp8_quant_weights(t((1, 16, 32)), out=(t((1, 16, 32), F8), t((1, 1, 1)),
                                                                                    None, None)),
    "moe_fp8_linear": lambda: moe.moe_fp8_linear(t((4, 32), F8), t((4, 1)), t((1, 16, 32), F8), t((1, 1, 1)),
                                                 out=t((4, 16), BF16)),
    "moe_fp8_linear_dw": lambda: moe.moe_fp8_linear_dw(t((16, 128), F8), t((16, 1)), t((32, 128), F8), t((32, 1)),
                                                       out=t((1, 16, 32), BF16)),
}


@pytest.fixture(params=["missing", "unloadable", "another library", "an older build"])
def without(request, monkeypatch):
    moe.lib()
    if request.param in ("another library", "an older build"):
        class Module:
            @staticmethod
            def init(*a):
                raise RuntimeError("the library lacks an entry point") if request.param == "another library" else \
                    TypeError("function takes exactly 2 arguments (3 given)")
        found = lambda *a: Module  # noqa: E731
    else:
        kind = ModuleNotFoundError if request.param == "missing" else ImportError

        def found(*a):
            raise kind("no _fast here")
    monkeypatch.setattr(moe, "_fast", None)
    monkeypatch.setattr(moe, "_lib", None)
    with monkeypatch.context() as m:
        m.setattr(moe.importlib, "import_module", found)
        with pytest.warns(RuntimeWarning, match="_fast"):
            moe.lib()


@pytest.mark.parametrize("name", CALLS)
def test_the_ordinary_way_answers(without, name):
    assert moe.moe_align_capacity(4, 2, 8, 16)
    with pytest.raises(moe.MoeError, match="must be on a GPU") as error:
        CALLS[name]()
    assert error.value.status == -2


LOAD = """
import sys, warnings
import torch
{before}
import mixture_experts_ffn_moe_amd as moe
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    moe.lib()
assert moe.moe_align_capacity(4, 2, 8, 16)
print("short way" if "_fast" in sys.modules.get("mixture_experts_ffn_moe_amd._fast", sys).__name__ else "ordinary way",
      *(str(w.message) for w in seen if "_fast" in str(w.message)))
"""


@pytest.mark.parametrize("before,way,word", [
    ("", "short way", ""), ("torch.__version__ = '1.13.0'", "ordinary way", "1.13.0"),
    ("torch.__version__ = torch.__version__ + '1'", "ordinary way", "torch")])
def test_another_torch(before, way, word):
    r = subprocess.run([sys.executable, "-c", LOAD.format(before=before)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith(way) and word in r.stdout
    assert (word == "") == (r.stdout.strip() == way)
