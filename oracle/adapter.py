"""Low-rank adapters beside the experts' products, one row at a time in 64 bits.

Every function takes the rows' experts and adapters (-1: none) and works on one row, or one (adapter, expert), after
the other; m is the matrix of dropout factors (or 1.0).
"""

import numpy as np


def row_groups(ids, offsets, row_token, n, L):
    """(expert [n], adapter [n]) of every row; expert -1 for rows behind the last expert's, adapter -1: none."""
    e, l = np.full(n, -1), np.full(n, -1)
    for x in range(len(offsets) - 1):
        e[offsets[x]:offsets[x + 1]] = x
    for r in range(n):
        t = r if row_token is None else row_token[r]
        if e[r] >= 0 and 0 <= t < len(ids) and 0 <= ids[t] < L:
            l[r] = ids[t]
    return e, l


def shrink(x, w, e, l, m=1.0):
    """(v [n, R], sum of magnitudes): v[r] = (m x)[r] W[l, e]^T, 0 without an adapter."""
    x = x * m
    v, mag = np.zeros((x.shape[0], w.shape[2])), np.zeros((x.shape[0], w.shape[2]))
    for r in np.flatnonzero(l >= 0):
        v[r], mag[r] = w[l[r], e[r]] @ x[r], np.abs(w[l[r], e[r]]) @ np.abs(x[r])
    return v, mag


def expand(v, w, e, l, scale=None):
    """(s v[r] W[l, e], sum of magnitudes), 0 without an adapter."""
    y, mag = np.zeros((v.shape[0], w.shape[3])), np.zeros((v.shape[0], w.shape[3]))
    for r in np.flatnonzero(l >= 0):
        s = 1.0 if scale is None else scale[l[r]]
        y[r], mag[r] = s * (v[r] @ w[l[r], e[r]]), abs(s) * (np.abs(v[r]) @ np.abs(w[l[r], e[r]]))
    return y, mag


def wgrad(v, y, e, l, shape, scale=None):
    """(dW [L, E, R, C], sum of magnitudes): v^T y over the rows of each adapter and expert."""
    dw, mag = np.zeros(shape), np.zeros(shape)
    for r in np.flatnonzero(l >= 0):
        s = 1.0 if scale is None else scale[l[r]]
        dw[l[r], e[r]] += s * np.outer(v[r], y[r])
        mag[l[r], e[r]] += abs(s) * np.outer(np.abs(v[r]), np.abs(y[r]))
    return dw, mag


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def forward(x, g, u, a_gu, b_gate, b_up, a_down, b_down, y, scale, e, l, m1=1.0, m2=1.0):
    """The whole of it without a rounding, for the pins: x by row; dict of v1, g, u, a, v2, y."""
    R = b_gate.shape[2]
    v1, _ = shrink(x, a_gu, e, l, m1)
    g = g + expand(v1[:, :R], b_gate, e, l, scale)[0]
    u = u + expand(v1[:, R:], b_up, e, l, scale)[0]
    a = g * sigmoid(g) * u
    v2, _ = shrink(a, a_down, e, l, m2)
    return dict(v1=v1, g=g, u=u, a=a, v2=v2, y=y + expand(v2, b_down, e, l, scale)[0])


def down_backward(dy, a, v2, a_down, b_down, scale, e, l, m2=1.0):
    """(da [n, f], d_a_down, d_b_down): what the adapters of the down product pass on and learn."""
    s = np.where(l >= 0, np.asarray(scale)[l], 0.0)[:, None]
    dv, _ = shrink(dy, b_down, e, l)
    dv = s * dv
    return (m2 * expand(dv, a_down, e, l)[0], wgrad(dv, a * m2, e, l, a_down.shape)[0],
            wgrad(v2, dy, e, l, b_down.shape, scale)[0])


def gate_up_backward(dg, du, x, v1, a_gu, b_gate, b_up, scale, e, l, m1=1.0):
    """(dx by row, d_a_gu, d_b_gate, d_b_up)."""
    R = b_gate.shape[2]
    s = np.where(l >= 0, np.asarray(scale)[l], 0.0)[:, None]
    dv = s * np.concatenate([shrink(dg, b_gate, e, l)[0], shrink(du, b_up, e, l)[0]], axis=1)
    return (m1 * expand(dv, a_gu, e, l)[0], wgrad(dv, x * m1, e, l, a_gu.shape)[0],
            wgrad(v1[:, :R], dg, e, l, b_gate.shape, scale)[0], wgrad(v1[:, R:], du, e, l, b_up.shape, scale)[0])
