"""Refusals of the products with 4-bit weights (CPU only)."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

from .test_rows_abi_cpu import Fake

P = ctypes.c_void_p
F, ODD = P(1 << 20), P((1 << 20) + 8)
NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4, -5


def matvec(fmt=0, elem=0, x=F, per=0, w=F, s=F, z=None, ids=F, out=F, T=2, K=256, N=64, E=4, k=2,
           group=128, swiglu=0):
    return moe.lib().moe_w4_matvec(fmt, elem, x, per, w, s, z, ids, out, T, K, N, E, k, group,
                                   swiglu, None)


def ffn(fmt=0, elem=0, x=F, w1=F, s1=F, z1=None, w2=F, s2=F, z2=None, ids=F, wt=F, out=F, T=2,
        K=256, N=256, E=4, k=2, group=128, ws=F, bytes_=1 << 30):
    return moe.lib().fused_moe_w4(fmt, elem, x, w1, s1, z1, w2, s2, z2, ids, wt, out, T, K, N, E,
                                  k, group, ws, bytes_, None)


@pytest.mark.parametrize("call", [matvec, ffn])
@pytest.mark.parametrize("bad,status", [
    (dict(fmt=2), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED), (dict(elem=2), UNSUPPORTED),
    (dict(elem=3), UNSUPPORTED), (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE),
    (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(group=-1), SHAPE), (dict(group=16), UNSUPPORTED),
    (dict(group=256, K=512, N=1024), UNSUPPORTED), (dict(K=192), UNSUPPORTED),
    (dict(K=192, group=0), UNSUPPORTED), (dict(fmt=1), UNSUPPORTED), (dict(T=2049), UNSUPPORTED),
    (dict(T=1 << 40), UNSUPPORTED), (dict(K=1 << 16, N=1 << 16), UNSUPPORTED),
    (dict(K=1 << 32), UNSUPPORTED), (dict(out=ODD), ALIGN), (dict(x=ODD), ALIGN), (dict(x=None), NULL),
    (dict(out=None), NULL)])
def test_sizes(call, bad, status):
    assert call(**bad) == status
    assert moe.lib().moe_last_error()


def test_matvec_arguments():
    assert matvec(ids=None) == NULL and matvec(ids=None, E=1) == NULL
    assert matvec(swiglu=1, N=63) == SHAPE
    assert matvec(fmt=1, group=32, z=F) == UNSUPPORTED
    for n in ("w", "s"):
        assert matvec(**{n: None}) == NULL and matvec(**{n: ODD}) == ALIGN
    assert matvec(z=ODD) == ALIGN and matvec(ids=ODD) == ALIGN
    assert matvec(T=0, x=None, ids=F, out=None) == 0


def test_ffn_arguments():
    assert ffn(N=255) == SHAPE
    assert ffn(N=192) == UNSUPPORTED          # I = 96 is no whole group
    assert ffn(fmt=1, group=32, z1=F) == UNSUPPORTED and ffn(fmt=1, group=32, z2=F) == UNSUPPORTED
    for n in ("w1", "s1", "w2", "s2", "ids", "wt"):
        assert ffn(**{n: None}) == NULL and ffn(**{n: ODD}) == ALIGN
    need = moe.moe_w4_workspace_size(2, 256, 256, 2)
    assert need >= 4 * 4 * (128 + 256)
    assert ffn(bytes_=need - 1) == WORKSPACE and ffn(ws=None) == WORKSPACE and ffn(ws=ODD) == ALIGN
    assert ffn(T=0, x=None, ids=None, wt=None, out=None, ws=None, bytes_=0) == 0


def test_workspace_errors():
    for args, status in (((-1, 256, 256, 2), SHAPE), ((2, 256, 255, 2), SHAPE),
                         ((4096, 256, 256, 2), UNSUPPORTED)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_w4_workspace_size(*args)
        assert e.value.status == status
    assert moe.moe_w4_workspace_size(0, 256, 256, 2) == 0


def test_binding_refuses():
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    x, ids, wt = Fake((2, 256)), Fake((2, 2), i32), Fake((2, 2), f32)
    w, s, z = Fake((4, 64, 128), u8), Fake((4, 64, 2)), Fake((4, 64, 2), u8)
    w.dim = ids.dim = x.dim = lambda: 3
    x.dim = ids.dim = lambda: 2
    flat = Fake((4 * 64, 128), u8)
    flat.dim = lambda: 2
    f = moe.moe_w4_matvec
    cases = [
        (UNSUPPORTED, lambda: f("int8", x, w, s, z, ids, 128)),
        (UNSUPPORTED, lambda: f("int4", Fake((2, 256), f32), w, s, z, ids, 128)),
        (SHAPE, lambda: f("int4", Fake((2, 256), cuda=False), w, s, z, ids, 128)),
        (SHAPE, lambda: f("int4", x, flat, s, z, ids, 128)),
        (SHAPE, lambda: f("int4", x, w, Fake((4, 64, 1)), z, ids, 128)),
        (UNSUPPORTED, lambda: f("int4", x, w, Fake((4, 64, 2), torch.float16), z, ids, 128)),
        (UNSUPPORTED, lambda: f("mx", x, w, Fake((4, 64, 8)), None, ids, 32)),
        (SHAPE, lambda: f("int4", x, w, s, Fake((4, 64, 1), u8), ids, 128)),
        (UNSUPPORTED, lambda: f("int4", x, w, s, Fake((4, 64, 2)), ids, 128)),
        (UNSUPPORTED, lambda: f("int4", x, w, s, z, Fake((2, 2), torch.int64), 128)),
        (SHAPE, lambda: f("int4", x, w, s, z, Fake((3, 2), i32), 128)),
        (SHAPE, lambda: f("int4", x, w, s, z, ids, 128, out=Fake((2, 2, 63)))),
        (SHAPE, lambda: f("int4", x, w, s, z, ids, 128, swiglu=True, out=Fake((2, 2, 64)))),
        (SHAPE, lambda: moe.fused_moe_w4("int4", x, w, s, z, Fake((4, 256, 32), u8), Fake((4, 256, 1)),
                                         None, ids, wt, 128)),
    ]
    for n, (status, call) in enumerate(cases):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == status, (n, str(e.value))


def test_binding_refuses_other_ranks():
    u8, i32 = torch.uint8, torch.int32
    w, s, ids = Fake((4, 64, 128), u8), Fake((4, 64, 2)), Fake((2, 2), i32)
    w.dim = lambda: 3
    for shape in ((), (256,), (1, 2, 2, 256)):
        x = Fake(shape)
        x.dim = lambda: len(shape)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_w4_matvec("int4", x, w, s, None, ids, 128)
        assert e.value.status == SHAPE
