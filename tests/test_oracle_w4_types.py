"""The 4-bit oracle's error model beside fp16 activations (CPU only): codes held
as q - 8 stay inside its bound, codes held as 1024 + q do not."""

import numpy as np
import pytest

from oracle import w4


def cancelling(group, zeros, N, K, T, rng):
    """Codes in pairs z + d, z - d, scales, zero points, and fp16 activations about 16: sums of large terms whose
    differences are the result."""
    n = K // group
    z = rng.integers(4, 12, (N, n)) if zeros else np.full((N, n), 8)
    q = np.empty((N, n, group), np.int64)
    d = rng.integers(-4, 5, (N, n, group // 2))
    q[:, :, 0::2], q[:, :, 1::2] = z[:, :, None] + d, z[:, :, None] - d
    q = q.reshape(N, K)
    w = (q[:, 0::2] | q[:, 1::2] << 4).astype(np.uint8)
    s = (rng.uniform(0.3, 1.5, (N, n)) / (5 * K ** 0.5)).astype(np.float16).astype(np.float64)
    x = (16 + rng.normal(size=(T, K))).astype(np.float16).astype(np.float64)
    return w, s, (z.astype(np.uint8) if zeros else None), x


def summed(w, s, z, group, x, offset):
    """The product as an fp32 sum over 32 elements at a time of codes held as q + offset."""
    f = np.float32
    q = w4.fp4_unpack(w).astype(np.float64) + offset
    z = (8.0 if z is None else z.astype(np.float64)) + offset
    out = np.zeros(len(w), f)
    for g in range(x.size // group):
        v, xs = np.zeros(len(w), f), f(0)
        for k in range(g * group, (g + 1) * group, 32):
            v = (v.astype(np.float64) + q[:, k:k + 32] @ x[k:k + 32]).astype(f)
            xs = f(float(xs) + x[k:k + 32].sum())
        zg = z if np.isscalar(z) else z[:, g]
        d = (v.astype(np.float64) - zg * float(xs)).astype(f)
        out = (out.astype(np.float64) + s[:, g] * d.astype(np.float64)).astype(f)
    return out.astype(np.float64)


@pytest.mark.parametrize("group,zeros", [(128, False), (128, True), (64, True), (32, True)])
def test_offset_of_fp16_codes(group, zeros):
    rng = np.random.default_rng(group)
    w, s, z, x = cancelling(group, zeros, 64, 512, 1, rng)
    parts, largest = w4.operands("int4", "f16")
    y, sigma = w4.product("int4", w, s, z, group, x[0], parts, largest)
    half = 2.0 ** -11 * np.abs(y)            # fp16's half step
    kept = np.abs(summed(w, s, z, group, x[0], -8) - y)
    lost = np.abs(summed(w, s, z, group, x[0], 1024) - y)
    assert (kept <= 6 * sigma).all()
    # past the model and the rounding of the result together
    assert (lost > 6 * sigma + half).mean() > 0.2
