"""Oracle of the products with 4-bit weights (test infrastructure, see the
package docstring).

Definition followed
-------------------
[DeepGEMM #411] "Summary" section: weights packed e2m1 with one e8m0 exponent
per 32 along K, as oracle.codecs decodes them.  The whole-number format has
codes q in 0..15 with a scale s and a zero point z for each group along K:
W = (q - z) s, z = 8 where none is given.  Two codes a byte, the even element
in the low nibble.

The error model is oracle.moe's for bf16 instructions: 32 products are added
with a zero-mean error of standard deviation u times their 2-norm, and every
fp32 addition and product rounds once, independently, u = 2^-24.  A whole-number
weight is held as 16 + q and the group's (16 + z) sum(x) is taken off again,
so both sums' errors scale with 31 (16 + 15), the largest weight held; beside
fp16 activations it is held as q - 8, and that largest one is 8.
Each function returns the value and one standard deviation of its error.
"""

import numpy as np

from .codecs import e2m1_decode, e8m0_decode, fp4_unpack

U = 2.0 ** -24
LARGEST = 16.0 + 15.0


def operands(fmt, elem):
    """(operands an activation of type ``elem`` is held as, largest whole-number
    weight held beside it)."""
    if elem == "f16":
        return (1, 8.0) if fmt == "int4" else (2, None)
    return 1, LARGEST


def dequant(fmt, w, scale, zero, group):
    """(N, K/2) bytes, (N, K/group) scales and zeros -> (N, K) fp64."""
    q = fp4_unpack(w)
    n = q.shape[1] // group
    q = q.reshape(len(q), n, group)
    if fmt == "mx":
        return (e2m1_decode(q) * e8m0_decode(scale)[:, :, None]).reshape(len(q), -1)
    z = 8.0 if zero is None else np.asarray(zero, np.float64)[:, :, None]
    s = np.asarray(scale, np.float64)[:, :, None]
    return ((q - z) * s).reshape(len(q), -1)


def product(fmt, w, scale, zero, group, x, parts, largest=LARGEST):
    """y = W x for one row x: (y, sigma), both (N,).  ``parts``: bf16 operands
    a value of x is held as, each an addition of its own; ``largest``: whole-number
    weight held (see operands)."""
    W = dequant(fmt, w, scale, zero, group)
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        y = W @ x
        terms2 = (W * W) @ (x * x)
    n = W.shape[1] // group
    span = np.abs(y) + 3 * np.sqrt(terms2)
    # the running sum: one addition per group (per 32 for the microscaling
    # format, where the instruction adds), its product with the scale, and
    # the waves' sums
    steps = (W.shape[1] // 32 if fmt == "mx" else n) * parts
    var = U * U * (terms2 + (steps + 12) * span ** 2)
    if fmt != "mx":
        xg = x.reshape(n, group)
        q = (xg * xg).sum(1)
        run = np.abs(xg.sum(1)) + 3 * np.sqrt(q)
        in_group = largest ** 2 * (q + (group // 32 * parts + 2) * run ** 2)
        var = var + 2 * U * U * (np.asarray(scale, np.float64) ** 2) @ in_group
    return y, np.sqrt(var)


def silu_mul(gate, up):
    """silu(gate) * up and its deviation, from (value, sigma) pairs."""
    (g, sg), (u, su) = gate, up
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-g))
    s = g * sig
    h = s * u
    slope = np.abs(sig * (1.0 + g * (1.0 - sig)))
    return h, np.sqrt((slope * u * sg) ** 2 + (s * su) ** 2) + (np.abs(g) + 6) * U * np.abs(h)


def ffn(fmt, W1, W2, group, x, ids, weights, parts):
    """The experts' FFN of every token: (out, sigma), both (T, K).  W1, W2:
    (codes, scales, zeros or None) of all experts."""
    T, k = ids.shape
    K = W2[0].shape[1]
    I = W1[0].shape[1] // 2
    g2 = group if group else I
    g1 = group if group else x.shape[1]
    out, var = np.zeros((T, K)), np.zeros((T, K))
    size = np.zeros((T, K))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < len(W1[0]):
                continue
            one = [None if v is None else v[e] for v in W1]
            two = [None if v is None else v[e] for v in W2]
            y, s = product(fmt, *one, g1, x[t], parts)
            h, sh = silu_mul((y[:I], s[:I]), (y[I:], s[I:]))
            y, s = product(fmt, *two, g2, h, 2)
            d = dequant(fmt, *two, g2)
            s2 = s ** 2 + (d * d) @ sh ** 2  # and what comes in with h
            w = float(weights[t, j])
            out[t] += w * y
            var[t] += w * w * s2
            size[t] += np.abs(w * y)
    return out, np.sqrt(var) + (k + 1) * U * size
