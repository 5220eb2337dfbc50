"""Refusals of the operators on the rows of a plan (CPU only): the C entries
reject bad arguments before anything is enqueued, the binding rejects tensors
that the kernels do not take."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe

P = ctypes.c_void_p
F = P(1 << 20)          # 16-byte aligned, never dereferenced (errors come first)
ODD = P((1 << 20) + 8)
NULL, SHAPE, UNSUPPORTED, ALIGN = -1, -2, -3, -4


def route_rows(ids=F, T=4, k=2, E=8, S=0, plan=F, ntp=F, cap=64, row=F):
    return moe.lib().moe_route_rows(ids, T, k, E, S, plan, ntp, cap, row, None)


def permute(elem=0, x=F, row=F, plan=F, ntp=F, rows=F, T=4, K=64, k=2, S=0, cap=64):
    return moe.lib().moe_permute(elem, x, row, plan, ntp, rows, T, K, k, S, cap, None)


def permute_backward(elem=0, d=F, row=F, dx=F, T=4, K=64, k=2, S=0, cap=64):
    return moe.lib().moe_permute_backward(elem, d, row, dx, T, K, k, S, cap, None)


def unpermute(elem=0, rows=F, row=F, w=F, out=F, T=4, K=64, k=2, S=0, cap=64):
    return moe.lib().moe_unpermute(elem, rows, row, w, out, T, K, k, S, cap, None)


def unpermute_backward(elem=0, g=F, rows=F, row=F, plan=F, ntp=F, w=F, d=F, dw=F, T=4, K=64, k=2,
                       S=0, cap=64):
    return moe.lib().moe_unpermute_backward(elem, g, rows, row, plan, ntp, w, d, dw, T, K, k, S,
                                            cap, None)


def route_backward(ids=F, w=F, dw=F, d=F, T=4, E=8, k=2):
    return moe.lib().moe_route_backward(ids, w, dw, d, T, E, k, None)


@pytest.mark.parametrize("call", [permute, permute_backward, unpermute, unpermute_backward])
@pytest.mark.parametrize("bad,status", [
    (dict(elem=4), UNSUPPORTED), (dict(elem=-1), UNSUPPORTED), (dict(T=-1), SHAPE),
    (dict(K=0), SHAPE), (dict(K=1 << 31), UNSUPPORTED), (dict(k=0), SHAPE), (dict(S=-1), SHAPE),
    (dict(T=1 << 30), SHAPE), (dict(T=1 << 40), SHAPE), (dict(cap=-1), SHAPE),
    (dict(cap=1 << 31), SHAPE), (dict(T=1 << 22, K=8192), UNSUPPORTED), (dict(row=ODD), ALIGN)])
def test_sizes(call, bad, status):
    assert call(**bad) == status
    assert moe.lib().moe_last_error()


@pytest.mark.parametrize("call,names", [
    (route_rows, ("ids", "plan", "row")), (permute, ("x", "row", "plan", "rows")),
    (permute_backward, ("d", "dx")), (unpermute, ("rows", "out")),
    (unpermute_backward, ("g", "rows", "row", "plan", "d")),
    (route_backward, ("ids", "w", "dw", "d"))])
def test_pointers(call, names):
    for n in names:
        assert call(**{n: None}) == NULL, n
        assert call(**{n: ODD}) == ALIGN, n


@pytest.mark.parametrize("call", [route_rows, permute, unpermute_backward])
def test_row_count_pointer(call):
    assert call(ntp=None) == NULL
    assert call(ntp=P((1 << 20) + 2)) == ALIGN


def test_bytes_are_moved_only():
    for call in (permute_backward, unpermute, unpermute_backward):
        assert call(elem=3) == UNSUPPORTED


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(E=1025), UNSUPPORTED),
    (dict(k=17), UNSUPPORTED), (dict(T=1 << 26), UNSUPPORTED)])
def test_route_backward_sizes(bad, status):
    assert route_backward(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(S=-1), SHAPE),
    (dict(T=1 << 31), SHAPE), (dict(cap=-1), SHAPE)])
def test_route_rows_sizes(bad, status):
    assert route_rows(**bad) == status


def test_empty_calls_launch_nothing():
    assert route_rows(T=0, ids=None, row=None, cap=0, plan=None) == 0
    assert permute(T=0, x=None, row=None, cap=0, plan=None, rows=None) == 0
    assert permute_backward(T=0, d=None, dx=None, cap=0) == 0
    assert unpermute(T=0, rows=None, out=None, cap=0) == 0
    assert unpermute_backward(T=0, g=None, rows=None, row=None, plan=None, d=None, cap=0) == 0
    assert route_backward(T=0, ids=None, w=None, dw=None, d=None) == 0


class Fake:
    """A tensor's face: what the binding looks at before it calls the library."""

    def __init__(self, shape, dtype=torch.bfloat16, dense=True, cuda=True, device="cuda:0"):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, cuda
        self.device = torch.device(device if cuda else "cpu")
        self.dense = dense

    def is_contiguous(self):
        return self.dense

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


def test_binding_refuses():
    i32, f32 = torch.int32, torch.float32
    x, row, plan, ntp = Fake((4, 64)), Fake((8,), i32), Fake((64,), i32), Fake((1,), i32)
    rows, w, ids = Fake((64, 64)), Fake((4, 2), f32), Fake((4, 2), i32)
    cases = [
        (SHAPE, lambda: moe.moe_permute(Fake((4, 64), cuda=False), row, plan, ntp, 2)),
        (UNSUPPORTED, lambda: moe.moe_permute(Fake((4, 64), torch.float64), row, plan, ntp, 2)),
        (SHAPE, lambda: moe.moe_permute(Fake((4, 64), dense=False), row, plan, ntp, 2)),
        (SHAPE, lambda: moe.moe_permute(x, row, plan, ntp, 3)),
        (UNSUPPORTED, lambda: moe.moe_permute(x, Fake((8,), torch.int64), plan, ntp, 2)),
        (SHAPE, lambda: moe.moe_permute(x, row, Fake((64,), i32, device="cuda:1"), ntp, 2)),
        (SHAPE, lambda: moe.moe_permute(x, row, plan, Fake((2,), i32), 2)),
        (SHAPE, lambda: moe.moe_permute(x, row, plan, ntp, 2, out=Fake((63, 64)))),
        (UNSUPPORTED, lambda: moe.moe_permute(x, row, plan, ntp, 2, out=Fake((64, 64), f32))),
        (SHAPE, lambda: moe.moe_permute_backward(rows, Fake((9,), i32), 2)),
        (SHAPE, lambda: moe.moe_unpermute(rows, row, Fake((4, 3), f32), 2)),
        (UNSUPPORTED, lambda: moe.moe_unpermute(rows, row, Fake((4, 2)), 2)),
        (SHAPE, lambda: moe.moe_unpermute(rows, row, w, 0)),
        (SHAPE, lambda: moe.moe_unpermute(rows, None, None, 3)),
        (SHAPE, lambda: moe.moe_unpermute_backward(x, Fake((60, 64)), row, plan, ntp, w, 2)),
        (UNSUPPORTED, lambda: moe.moe_unpermute_backward(x, Fake((64, 64), f32), row, plan, ntp, w, 2)),
        (SHAPE, lambda: moe.moe_route_rows(Fake((4, 2), i32, cuda=False), 8, plan, ntp)),
        (UNSUPPORTED, lambda: moe.moe_route_rows(Fake((4, 2), torch.int64), 8, plan, ntp)),
        (SHAPE, lambda: moe.moe_route_backward(ids, w, Fake((4, 3), f32), 8)),
        (SHAPE, lambda: moe.moe_route_backward(ids, w, w, 8, out=Fake((4, 9), f32))),
    ]
    for n, (status, call) in enumerate(cases):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == status, (n, str(e.value))


def test_one_launch_holds_the_call():
    # four tokens a workgroup, and a launch has less than 2^24 of them
    assert route_backward(T=(1 << 26) - 3) == UNSUPPORTED
    assert b"2^26" in moe.lib().moe_last_error()


def test_binding_refuses_negative_counts():
    i32, f32 = torch.int32, torch.float32
    plan, ntp, ids, w = Fake((64,), i32), Fake((1,), i32), Fake((4, 2), i32), Fake((4, 2), f32)
    for call in (lambda: moe.moe_route_rows(ids, 8, plan, ntp, n_shared=-3),
                 lambda: moe.moe_route_backward(ids, w, w, -1)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == SHAPE
