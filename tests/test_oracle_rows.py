"""Pins of the rows oracle (CPU only): a hand case, adjointness of the forward
and backward maps, and the router's gradient against differences of the
router oracle's weights."""

import numpy as np
import pytest

from oracle.align import align_ref
from oracle.router import route_ref
from oracle.rows import (permute_ref, route_backward_ref, route_rows_ref, unpermute_backward_ref,
                         unpermute_ref)


def test_hand_case():
    # two tokens, two routes each over 2 experts of block 2; token 1's second
    # route is elsewhere (expert 5)
    ids = np.array([[1, 0], [1, 5]])
    plan, _, ntp = align_ref(ids, 2, 2)
    assert ntp == 4 and plan[:4].tolist() == [1, -1, 0, 2]
    row = route_rows_ref(plan, ntp, 4)
    assert row.tolist() == [2, 0, 3, -1]
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    rows = permute_ref(x, plan, ntp, 2)
    assert rows.tolist() == [[1, 2], [0, 0], [1, 2], [3, 4]]
    w = np.array([[0.25, 0.75], [0.5, 0.5]])
    out, mag = unpermute_ref(np.array([[8.0, 0], [9, 9], [4, 4], [2, -2]]), plan, ntp, w, 2, 2)
    assert out.tolist() == [[7, 1], [1, -1]] and mag.tolist() == [[7, 1], [1, 1]]
    d_rows, d_w, _ = unpermute_backward_ref(np.array([[1.0, 1], [2, 0]]), rows, plan, ntp, w, 2, 2)
    assert d_rows.tolist() == [[0.75, 0.75], [0, 0], [0.25, 0.25], [1, 0]]
    assert d_w.tolist() == [[3, 3], [6, 0]]


@pytest.mark.parametrize("n_shared", [0, 2])
def test_backward_is_the_adjoint(n_shared):
    rng = np.random.default_rng(5)
    T, k, E, K, bm = 7, 3, 4, 5, 4
    routed = np.array([rng.permutation(E + 1)[:k] for _ in range(T)])
    flat = np.full(T * (k + n_shared), -1)
    flat[:T * k] = np.where(routed < E, routed, -1).reshape(-1)
    for s in range(n_shared):
        flat[T * k + np.arange(T) * n_shared + s] = E + s
    plan, _, ntp = align_ref(flat.reshape(-1, 1), E + n_shared, bm)
    x, y, g = rng.normal(size=(T, K)), rng.normal(size=(len(plan), K)), rng.normal(size=(T, K))
    w = rng.random((T, k))
    # <permute(x), y> = <x, permute_backward(y)>
    back, _ = unpermute_ref(y, plan, ntp, None, T, k, n_shared)
    assert np.isclose((permute_ref(x, plan, ntp, k, n_shared) * y[:ntp]).sum(), (x * back).sum())
    # the weighted sum is linear in the rows and in the weights
    out, _ = unpermute_ref(y, plan, ntp, w, T, k, n_shared)
    d_rows, d_w, _ = unpermute_backward_ref(g, y, plan, ntp, w, T, k, n_shared)
    assert np.isclose((d_rows * y[:ntp]).sum(), (g * out).sum())
    shared, _ = unpermute_ref(y, plan, ntp, np.zeros_like(w), T, k, n_shared)
    assert np.isclose((d_w * w).sum(), (g * (out - shared)).sum())


def test_route_backward_against_differences():
    rng = np.random.default_rng(6)
    T, E, k, step = 5, 9, 4, 1e-6
    L, g = rng.normal(size=(T, E)), rng.normal(size=(T, k))
    ids, w = route_ref(L, k)
    d = route_backward_ref(ids, w, g, E)
    for t in range(T):
        for e in range(E):
            up, down = L.copy(), L.copy()
            up[t, e] += step
            down[t, e] -= step
            (iu, wu), (il, wl) = route_ref(up, k), route_ref(down, k)
            assert (iu == ids).all() and (il == ids).all()
            num = ((wu - wl)[t] * g[t]).sum() / (2 * step)
            # central differences: step^2 / 6 times a third derivative of
            # order one, plus 2^-53 / step of rounding
            assert abs(num - d[t, e]) < 1e-9 * 10


def test_planted_mistakes_fail():
    """A weight left out, and a gradient without the softmax's mean, differ."""
    rng = np.random.default_rng(7)
    ids = np.array([rng.permutation(6)[:2] for _ in range(4)])
    plan, _, ntp = align_ref(ids, 6, 4)
    y, w = rng.normal(size=(len(plan), 3)), rng.random((4, 2))
    assert not np.allclose(unpermute_ref(y, plan, ntp, w, 4, 2)[0],
                           unpermute_ref(y, plan, ntp, None, 4, 2)[0])
    L, g = rng.normal(size=(4, 6)), rng.normal(size=(4, 2))
    i, wr = route_ref(L, 2)
    d = route_backward_ref(i, wr, g, 6)
    assert not np.allclose(np.take_along_axis(d, i.astype(int), 1), wr * g)
