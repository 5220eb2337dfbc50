"""Pins of the 8-bit linear layers' oracle (CPU only)."""

import numpy as np
import pytest

from oracle.codecs import e4m3_decode
from oracle.fp8 import block_values, product, quant_blocks, quant_columns, quant_rows, row_values, scale_values


def test_hand_case():
    x = np.zeros((1, 256), np.float32)
    x[0, 0], x[0, 1], x[0, 128] = 896.0, -2.0, 1.75
    q, s = quant_rows(x, "f32")
    assert np.allclose(s, [[2.0, 1.75 / 448]], rtol=1e-7)
    assert e4m3_decode(q)[0, [0, 1, 128]].tolist() == [448, -1, 448]
    q, s = quant_rows(x, "e8m0")
    # 896 = 448 * 2; 1.75 = 448 * 2^-8 exactly
    assert s.tolist() == [[128, 119]] and e4m3_decode(q)[0, [0, 1, 128]].tolist() == [448, -1, 448]
    # the next value up takes the next power of two
    x[0, 128] = np.nextafter(np.float32(1.75), np.float32(2))
    assert quant_rows(x, "e8m0")[1].tolist() == [[128, 120]]
    # nothing: the floor's scale, and zeros
    q, s = quant_rows(np.zeros((1, 16), np.float32), "e8m0")
    assert not q.any() and 448 * scale_values(s)[0, 0] >= 1e-30 > 224 * scale_values(s)[0, 0]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_errors_and_layouts(kind):
    rng = np.random.default_rng(1)
    x = (rng.normal(size=(200, 144)) * np.exp(3 * rng.normal(size=(200, 1)))).astype(np.float32)
    step = {"f32": 2.0 ** -9 / 448, "e8m0": 2.0 ** -9 / 224}[kind]  # half a subnormal step, of amax
    for values, amax in ((row_values(*quant_rows(x, kind)), None), (block_values(*quant_blocks(x, kind)), None)):
        assert (np.abs(values - x) <= 2.0 ** -4 * np.abs(x) * (1 + 1e-6) + step * np.abs(x).max()).all()
    q, s = quant_columns(x, kind)
    assert q.shape == (144, 256) and s.shape == (144, 2) and not q[:, 200:].any()
    assert np.array_equal(q[:, :128], quant_rows(np.ascontiguousarray(x[:128].T), kind)[0])


def test_product():
    rng = np.random.default_rng(2)
    x, w = rng.integers(-3, 4, (5, 300)).astype(float), rng.integers(-3, 4, (7, 300)).astype(float)
    y, sigma = product(x, w)
    assert y[2, 3] == sum(a * b for a, b in zip(x[2], w[3]))
    assert (sigma >= 2.0 ** -15 * np.sqrt((x * x) @ (w * w).T)).all()
