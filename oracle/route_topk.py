"""General router oracle: scores, a bias for the choice, groups, top-k, weights,
and the gradient of the weights.  fp64 from the logits as they are given.

The pages leave the gate to the caller ([prime-flash] "Usage"); the definition is
the C ABI's (moe_route_topk): s the softmax or the sigmoid of the unmasked
logits, c = s + bias chooses, first the groups (the sum of a group's group_top
largest c, fewer where it has fewer), then the experts; ties go to the lower
index; ids are -1 and weights 0 where no candidate is left.
"""

import math

import numpy as np

LARGEST = float(np.finfo(np.float32).max)


def _clean(logits):
    L = np.array(logits, dtype=np.float64)
    L[np.isnan(L)] = -np.inf
    return np.minimum(L, LARGEST)


def scores(logits, scoring):
    """s of every expert, 0 where masked."""
    L = _clean(logits)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-L))
    m = L.max(axis=1, keepdims=True)
    e = np.exp(L - np.where(np.isinf(m), 0.0, m))
    total = e.sum(axis=1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def _largest(values, n):
    """Indices of the n largest, largest first, ties to the lower."""
    return sorted(range(len(values)), key=lambda i: (-values[i], i))[:n]


def chosen_weights(logits, ids, scoring, renormalize, scale):
    """Weights of given ids (-1: none).  Renormalized softmax weights are the
    softmax over the chosen logits, which holds also where the others dwarf them."""
    L, s = _clean(logits), scores(logits, scoring)
    w = np.zeros(ids.shape)
    for t in range(ids.shape[0]):
        at = [j for j in range(ids.shape[1]) if ids[t, j] >= 0]
        if not at:
            continue
        v = s[t, ids[t, at]]
        if renormalize and scoring == "softmax":
            l = L[t, ids[t, at]]
            v = np.exp(l - l.max()) if l.max() > -np.inf else np.zeros(len(at))
        if renormalize:
            v = v / v.sum() if v.sum() > 0 else 0.0 * v
        w[t, at] = v * scale
    return w


def route_topk_ref(logits, top_k, bias=None, scoring="softmax", n_group=1, topk_group=1, group_top=1,
                   renormalize=True, scale=1.0):
    """(ids (T, top_k) int32, weights (T, top_k) float64)."""
    L = _clean(logits)
    T, E = L.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    c = scores(logits, scoring) + b
    c[(L == -np.inf) | np.isnan(c)] = -np.inf
    size = E // n_group
    ids = np.full((T, top_k), -1, np.int32)
    for t in range(T):
        total = []
        for g in range(n_group):
            best = sorted((v for v in c[t, g * size:(g + 1) * size] if v > -math.inf), reverse=True)[:group_top]
            total.append(sum(best) if best else -math.inf)
        kept = _largest(total, topk_group)
        left = [e for e in range(E) if e // size in kept and c[t, e] > -math.inf]
        pick = _largest([c[t, e] for e in left], top_k)
        ids[t, :len(pick)] = [left[i] for i in pick]
    return ids, chosen_weights(logits, ids, scoring, renormalize, scale)


def route_topk_backward_ref(logits, ids, d_weights, scoring, renormalize, scale):
    """d_logits (T, E) by the chain rule, written with full Jacobians."""
    L, s = _clean(logits), scores(logits, scoring)
    T, E = L.shape
    out = np.zeros((T, E))
    for t in range(T):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not at:
            continue
        e, g = ids[t, at], np.asarray(d_weights, np.float64)[t, at] * scale
        if scoring == "softmax" and renormalize:
            l = L[t, e]
            if l.max() == -np.inf:
                continue
            p = np.exp(l - l.max())
            p /= p.sum()
            np.add.at(out[t], e, (np.diag(p) - np.outer(p, p)) @ g)
            continue
        v = s[t, e]
        if renormalize:
            S = v.sum()
            if S == 0:
                continue
            g = (np.eye(len(at)) - np.outer(np.ones(len(at)), v / S)) @ g / S  # (S squared may be 0)
        ds = np.zeros(E)
        np.add.at(ds, e, g)
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                out[t] = ds * s[t] * (1.0 / (1.0 + np.exp(L[t])))
        else:
            out[t] = (np.diag(s[t]) - np.outer(s[t], s[t])) @ ds
    return out
