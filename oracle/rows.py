"""Rows between token order and expert order, in float64.

Test infrastructure (see the package docstring).  Pair (t, j) stands at row inv[t, j]; places
outside [0, n) are dropped pairs.
"""
from __future__ import annotations

import numpy as np


def _pairs(inv, n):
    for t, j in np.ndindex(*inv.shape):
        if 0 <= inv[t, j] < n:
            yield t, j, inv[t, j]


def dispatch(x, inv, n, rows):
    """rows with x's rows at the places of their pairs (the rest as it was)."""
    rows = rows.copy()
    for t, _, at in _pairs(inv, n):
        rows[at] = x[t]
    return rows


def combine(y, inv, n, w=None, residual=None):
    """Each token's rows, weighted, summed onto the residual; and the sum of the magnitudes."""
    out = np.zeros((inv.shape[0], y.shape[1])) if residual is None else residual.astype(np.float64)
    mag = np.abs(out)
    for t, j, at in _pairs(inv, n):
        term = y[at] * (1.0 if w is None else float(w[t, j]))
        out[t] = out[t] + term
        mag[t] = mag[t] + np.abs(term)
    return out, mag


def combine_grad(dout, y, inv, n, w, dy):
    """dy (the rest as it was), the routing weights' gradient and the magnitudes of its terms."""
    dy, dw, mag = dy.copy(), np.zeros(inv.shape), np.zeros(inv.shape)
    for t, j, at in _pairs(inv, n):
        dy[at] = dout[t] * (1.0 if w is None else float(w[t, j]))
        if y is not None:
            dw[t, j] = np.dot(dout[t], y[at])
            mag[t, j] = np.dot(np.abs(dout[t]), np.abs(y[at]))
    return dy, dw, mag
