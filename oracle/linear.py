"""The dense product with its epilogue and its gradients, in float64.

Test infrastructure (see the package docstring).
"""
from __future__ import annotations

import numpy as np

C = np.sqrt(2.0 / np.pi)


def sigmoid(t):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t))


def _half(v):
    """(1 + tanh(u)) / 2 of tanh-GELU, u = C (v + 0.044715 v^3), as the sigmoid of 2 u, which
    loses nothing where tanh is near -1."""
    return sigmoid(2.0 * C * (v + 0.044715 * v ** 3))


def act(v, name):
    if name == "none":
        return v
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return v * sigmoid(v)
    return v * _half(v)


def act_grad(v, name):
    if name == "none":
        return np.ones_like(v)
    if name == "relu":
        return (v > 0).astype(np.float64)
    if name == "silu":
        s = sigmoid(v)
        return s + v * s * (1.0 - s)
    s = _half(v)
    return s + v * s * (1.0 - s) * 2.0 * C * (1.0 + 3 * 0.044715 * v * v)


def product(x, w):
    """x w^T and the sums of the products' magnitudes."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def fwd(x, w, bias, name, residual):
    """(y, z, magnitudes of z's terms)"""
    z, mag = product(x, w)
    if bias is not None:
        z, mag = z + bias, mag + np.abs(bias)
    y = act(z, name)
    return (y if residual is None else y + residual), z, mag


def dgrad(dz, w, zx, name, add):
    """(dx, dz w, magnitudes of its terms)"""
    d, mag = product(dz, np.ascontiguousarray(w.T))
    dx = d if name == "none" else d * act_grad(zx, name)
    return (dx if add is None else dx + add), d, mag


def wgrad(dz, x):
    """(dw, magnitudes, db, magnitudes)"""
    a, b = np.ascontiguousarray(dz.T), np.ascontiguousarray(x.T)
    return (*product(a, b), dz.sum(0), np.abs(dz).sum(0))
