"""8-bit linear layers' oracle: quantizers into e4m3 with a scale per 128, and
products of such values in fp64.

Readings: a group's scale is amax / 448 held in fp32 (as fp32(amax * fp32(1 /
448)), values times fp32(1 / scale): the precision in which [DeepGEMM #88]
"Before you merge" states the forward's requantization), or the smallest power of
two at or above amax / 448.  amax is floored at 1e-30.
"""

import numpy as np

from .codecs import e4m3_decode, e4m3_encode, e8m0_decode

# the matrix instruction's error for one 128-wide step, relative to the products'
# 2-norm (twice the measured RMS), and fp32's half step
KAPPA = 2.0 ** -15
U = 2.0 ** -24
FLOOR = np.float32(1e-30)


def _scale(amax, kind):
    """(scale as held, the fp32 factor) of one group."""
    a = np.float32(max(np.float32(amax), FLOOR))
    if kind == "f32":
        s = np.float32(a * np.float32(1.0 / 448.0))
        return s, np.float32(1.0) / s
    e = -126
    while 448.0 * 2.0 ** e < float(a):
        e += 1
    while 448.0 * 2.0 ** (e - 1) >= float(a):
        e -= 1
    return np.uint8(e + 127), np.float32(2.0 ** -e)


def _held(kind):
    return np.float32 if kind == "f32" else np.uint8


def quant_rows(x, kind):
    """x (M, K) float32 -> codes (M, K), scales (M, ceil(K / 128))."""
    M, K = x.shape
    G = -(-K // 128)
    q, s = np.zeros((M, K), np.uint8), np.zeros((M, G), _held(kind))
    for m in range(M):
        for g in range(G):
            v = x[m, 128 * g:128 * g + 128]
            s[m, g], f = _scale(np.abs(v).max(), kind)
            q[m, 128 * g:128 * g + 128] = e4m3_encode((v * f).astype(np.float64))
    return q, s


def quant_columns(x, kind):
    """x (M, K) -> codes (K, Mp), scales (K, Mp / 128), zeros behind M."""
    M, K = x.shape
    p = np.zeros((K, -(-M // 128) * 128), np.float32)
    p[:, :M] = x.T
    return quant_rows(p, kind)


def quant_blocks(w, kind):
    """w (N, K) -> codes, scales (ceil(N / 128), ceil(K / 128))."""
    N, K = w.shape
    q = np.zeros((N, K), np.uint8)
    s = np.zeros((-(-N // 128), -(-K // 128)), _held(kind))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            s[i, j], f = _scale(np.abs(w[at]).max(), kind)
            q[at] = e4m3_encode((w[at] * f).astype(np.float64))
    return q, s


def scale_values(s):
    return e8m0_decode(s) if s.dtype == np.uint8 else s.astype(np.float64)


def row_values(q, s):
    return e4m3_decode(q) * np.repeat(scale_values(s), 128, axis=1)[:, :q.shape[1]]


def block_values(q, s):
    f = np.repeat(np.repeat(scale_values(s), 128, axis=0), 128, axis=1)
    return e4m3_decode(q) * f[:q.shape[0], :q.shape[1]]


def product(x, w):
    """(x @ w.T, the standard deviation of a correct kernel's result around it):
    the instruction's steps, and fp32 additions and scale products of the running
    sum, independent between steps.  For products of like size: the instruction
    cuts each off below 2^-13 of the largest of its eight, so that where one of
    eight outweighs the rest a step is off by up to 7 2^-13 of that one."""
    y = x @ w.T
    norm2 = (x * x) @ (w * w).T
    steps = -(-x.shape[1] // 128)
    add = U * np.sqrt(steps + 2) * (np.abs(y) + 3 * np.sqrt(norm2))
    return y, np.sqrt(KAPPA ** 2 * norm2 + add ** 2)
