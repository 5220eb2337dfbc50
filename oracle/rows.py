"""Oracle of the rows of a plan: tokens into the plan's rows and back, the
gradients of both, and the router's gradient.

Test infrastructure (see the package docstring).

Definition followed
-------------------
[hpc-ops RFC] "Background" section: the forward gathers the routed tokens and
ends with the top-k weighted reduction; [prime-flash] "Shapes" section: row p of
a plan holds the flat route id sorted_token_ids[p] or -1.  The gradients are
those two maps' adjoints, and the derivative of the normalized softmax weights.

Route ids: t * top_k + j for the routed ones, then T * top_k + t * S + s for
S shared experts.  All in fp64 from exact inputs, one loop per row, so that
nothing is shared with the way the kernels walk the tokens.
"""

import numpy as np


def token_of(r, T, top_k, n_shared=0):
    return r // top_k if r < T * top_k else (r - T * top_k) // n_shared


def placed(sorted_ids, ntp):
    """(row, route) pairs of the rows in use that hold a route."""
    return [(p, int(sorted_ids[p])) for p in range(int(ntp)) if sorted_ids[p] >= 0]


def route_rows_ref(sorted_ids, ntp, n_routes):
    row = np.full(n_routes, -1, np.int32)
    for p, r in placed(sorted_ids, ntp):
        row[r] = p
    return row


def permute_ref(x, sorted_ids, ntp, top_k, n_shared=0):
    """The rows below ntp: (ntp, K) fp64."""
    x = np.asarray(x, np.float64)
    out = np.zeros((int(ntp), x.shape[1]))
    for p, r in placed(sorted_ids, ntp):
        out[p] = x[token_of(r, len(x), top_k, n_shared)]
    return out


def unpermute_ref(rows, sorted_ids, ntp, weights, T, top_k, n_shared=0):
    """(out, sum of the terms' magnitudes), both (T, K) fp64; weights (T,
    top_k) or None for ones."""
    out = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(out)
    for p, r in placed(sorted_ids, ntp):
        w = 1.0
        if weights is not None and r < T * top_k:
            w = float(weights[r // top_k, r % top_k])
        y = w * np.asarray(rows[p], np.float64)
        t = token_of(r, T, top_k, n_shared)
        out[t] += y
        mag[t] += np.abs(y)
    return out, mag


def unpermute_backward_ref(d_out, rows, sorted_ids, ntp, weights, T, top_k, n_shared=0):
    """(d_rows below ntp, d_weights, sum of the dot products' term magnitudes)."""
    d_out = np.asarray(d_out, np.float64)
    d_rows = np.zeros((int(ntp), d_out.shape[1]))
    d_w = np.zeros((T, top_k))
    mag = np.zeros((T, top_k))
    for p, r in placed(sorted_ids, ntp):
        t = token_of(r, T, top_k, n_shared)
        w = 1.0
        if r < T * top_k:
            if weights is not None:
                w = float(weights[r // top_k, r % top_k])
            if rows is not None:
                prod = np.asarray(rows[p], np.float64) * d_out[t]
                d_w[r // top_k, r % top_k] = prod.sum()
                mag[r // top_k, r % top_k] = np.abs(prod).sum()
        d_rows[p] = w * d_out[t]
    return d_rows, d_w, mag


def route_backward_ref(ids, weights, d_weights, E):
    """(T, E) fp64 gradient of the logits, from the softmax's Jacobian
    dw_i / dl_j = w_i (delta_ij - w_j) over the selection."""
    w = np.asarray(weights, np.float64)
    g = np.asarray(d_weights, np.float64)
    T, k = w.shape
    out = np.zeros((T, E))
    for t in range(T):
        jac = np.diag(w[t]) - np.outer(w[t], w[t])
        for j in range(k):
            if 0 <= ids[t][j] < E:
                out[t, ids[t][j]] += float(g[t] @ jac[:, j])
    return out
