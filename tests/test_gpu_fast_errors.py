"""A launch that fails in the short way into the library raises, as it does in the
ordinary one: it is not made again.  (A stub in place of the library fails once; it
touches no GPU.)"""

import ctypes
import shutil
import subprocess

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

pytestmark = pytest.mark.gpu

ENTRIES = ("moe_route_topk", "moe_route_topk_backward", "moe_fp8_quant", "moe_fp8_quant_weights", "moe_fp8_linear",
           "moe_fp8_linear_dw")
STUB = "static int status, calls;\nvoid fail_once(int s) { status = s; calls = 0; }\nint count(void) { return calls; }\n" \
    "int hipGetDevice(int *d) { *d = 0; return 0; }\n" + "".join(
        f"int {name}(void) {{ int s = status; status = 0; ++calls; return s; }}\n" for name in ENTRIES)

F8 = torch.float8_e4m3fn


def v(shape, dtype=torch.float32):
    return torch.ones(shape, device="cuda").to(dtype)


def calls():
    i32 = torch.int32
    l, ids, w = v((4, 16)), torch.zeros(4, 2, dtype=i32, device="cuda"), v((4, 2))
    x, q, s = v((4, 32)), v((4, 32), F8), v((4, 1))
    wq, ws = v((1, 16, 32), F8), v((1, 1, 1))
    t, ts = v((16, 128), F8), v((16, 1))
    return {
        "moe_route_topk": lambda: moe.moe_route_topk(l, 2, out=(ids, w)),
        "moe_route_topk_backward": lambda: moe.moe_route_topk_backward(l, ids, w, out=v((4, 16))),
        "moe_fp8_quant": lambda: moe.moe_fp8_quant(x, out=(q, s, None, None)),
        "moe_fp8_quant_weights": lambda: moe.moe_fp8_quant_weights(v((1, 16, 32)), out=(wq, ws, None, None)),
        "moe_fp8_linear": lambda: moe.moe_fp8_linear(q, s, wq, ws, out=v((4, 16), torch.bfloat16)),
        "moe_fp8_linear_dw": lambda: moe.moe_fp8_linear_dw(t, ts, t, ts, out=v((1, 16, 16), torch.bfloat16)),
    }


@pytest.fixture
def stub(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("needs a C compiler")
    src, lib = tmp_path / "stub.c", tmp_path / "stub.so"
    src.write_text(STUB)
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    made = calls()  # tensors, and the library itself, before the stub takes its place
    moe.lib()
    stub = ctypes.CDLL(str(lib))
    moe._short_way(stub)
    try:
        yield stub, made
    finally:
        moe._short_way(moe.lib())


@pytest.mark.parametrize("name", ENTRIES)
def test_a_failed_launch_raises(stub, name):
    lib, made = stub
    lib.fail_once(-6)
    with pytest.raises(moe.MoeError) as error:
        made[name]()
    assert error.value.status == -6 and lib.count() == 1
    # and the next call is an ordinary one
    made[name]()
    assert lib.count() == 2


@pytest.mark.parametrize("name", ENTRIES)
def test_refused_arguments_are_worded_by_the_ordinary_way(stub, name):
    # nothing was enqueued: the ordinary way looks, here finds nothing wrong, and makes the call
    lib, made = stub
    lib.fail_once(-2)
    made[name]()
    assert lib.count() == 1
    torch.cuda.synchronize()
