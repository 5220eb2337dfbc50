"""Pins of the 4-bit oracle (CPU only): hand cases, a brute-force product, the
FFN against a plain one, and planted mistakes."""

import numpy as np

from oracle import w4


def test_hand_cases():
    w = np.full((1, 16), 0x88, np.uint8)
    w[0, 0] = 0x9F                       # element 0: code 15, element 1: code 9
    s = np.array([[0.5]])
    d = w4.dequant("int4", w, s, None, 32)
    assert d[0, 0] == 3.5 and d[0, 1] == 0.5 and not d[0, 2:].any()
    d = w4.dequant("int4", w, s, np.array([[15]]), 32)
    assert d[0, 0] == 0.0 and d[0, 1] == -3.0 and (d[0, 2:] == -3.5).all()
    d = w4.dequant("mx", w, np.array([[128]]), None, 32)
    # code 15: -6, code 9: -0.5, code 8: -0, times 2
    assert d[0, 0] == -12.0 and d[0, 1] == -1.0 and not d[0, 2:].any()


def test_product_by_loops():
    rng = np.random.default_rng(3)
    for fmt, group in (("int4", 32), ("int4", 64), ("mx", 32)):
        w = rng.integers(0, 256, (5, 64), dtype=np.uint8)
        n = 128 // group
        s = rng.integers(120, 130, (5, n)) if fmt == "mx" else rng.random((5, n))
        z = None if fmt == "mx" else rng.integers(0, 16, (5, n))
        x = rng.normal(size=128)
        y, sigma = w4.product(fmt, w, s, z, group, x, 1)
        mags = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
        for r in range(5):
            total = 0.0
            for k in range(128):
                q = (int(w[r, k // 2]) >> (4 * (k % 2))) & 15
                if fmt == "mx":
                    v = mags[q & 7] * (-1 if q > 7 else 1) * 2.0 ** (int(s[r, k // 32]) - 127)
                else:
                    v = (q - int(z[r, k // group])) * s[r, k // group]
                total += v * x[k]
            assert abs(total - y[r]) < 1e-12
        assert (sigma > 0).all()


def _ffn_inputs(rng, E=3, I=32, K=64):
    W1 = (rng.integers(0, 256, (E, 2 * I, K // 2), dtype=np.uint8), rng.random((E, 2 * I, K // 32)) / 40, None)
    W2 = (rng.integers(0, 256, (E, K, I // 2), dtype=np.uint8), rng.random((E, K, I // 32)) / 40, None)
    return W1, W2


def test_ffn_against_a_plain_one():
    rng = np.random.default_rng(4)
    W1, W2 = _ffn_inputs(rng)
    x, w = rng.normal(size=(4, 64)), rng.random((4, 2))
    ids = np.array([[0, 1], [2, 7], [-1, 1], [1, 1]])
    out, sigma = w4.ffn("int4", W1, W2, 32, x, ids, w, 1)
    D1 = [w4.dequant("int4", W1[0][e], W1[1][e], None, 32) for e in range(3)]
    D2 = [w4.dequant("int4", W2[0][e], W2[1][e], None, 32) for e in range(3)]
    for t in range(4):
        want = np.zeros(64)
        for j in range(2):
            e = ids[t, j]
            if 0 <= e < 3:
                g, u = np.split(D1[e] @ x[t], 2)
                want += w[t, j] * (D2[e] @ (g / (1 + np.exp(-g)) * u))
        assert np.allclose(out[t], want, rtol=1e-12, atol=1e-14)
    assert (sigma > 0).all()


def test_planted_mistakes_fail():
    """Swapped nibbles, a zero point left out, gate and up exchanged."""
    rng = np.random.default_rng(5)
    W1, W2 = _ffn_inputs(rng)
    x, w, ids = rng.normal(size=(2, 64)), np.ones((2, 1)), np.array([[0], [2]])
    out, sigma = w4.ffn("int4", W1, W2, 32, x, ids, w, 1)
    swap = lambda b: ((b << 4) | (b >> 4)).astype(np.uint8)                     # noqa: E731
    flip = tuple(None if v is None else np.concatenate(np.split(v, 2, 1)[::-1], 1) for v in W1)
    ones = np.full(W1[1].shape, 9)
    for bad in ((swap(W1[0]), W1[1], None), flip, (W1[0], W1[1], ones)):
        got, _ = w4.ffn("int4", bad, W2, 32, x, ids, w, 1)
        assert (np.abs(got - out) > 100 * sigma).any()
