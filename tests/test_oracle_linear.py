"""Pins of oracle/linear.py and oracle/rows.py: loops over scalars, the tanh form of the GELU, and
differences."""
import math

import numpy as np
import pytest

from oracle import linear, rows

ACTS = ["none", "relu", "silu", "gelu_tanh"]


def scalar_act(v, name):
    if name == "none":
        return v
    if name == "relu":
        return max(v, 0.0)
    if name == "silu":
        return v / (1 + math.exp(-v))
    return 0.5 * v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


@pytest.mark.parametrize("name", ACTS)
def test_activations(name):
    v = np.concatenate([np.linspace(-6, 6, 601), [-30.0, 30.0]])
    assert np.allclose(linear.act(v, name), [scalar_act(x, name) for x in v], rtol=1e-12, atol=1e-14)
    h = 1e-5
    d = (linear.act(v + h, name) - linear.act(v - h, name)) / (2 * h)
    keep = np.abs(v) > h if name == "relu" else np.ones_like(v, dtype=bool)
    assert np.allclose(linear.act_grad(v, name)[keep], d[keep], atol=1e-8)
    assert linear.act_grad(np.zeros(1), "relu")[0] == 0


def test_product_and_gradients():
    rng = np.random.default_rng(0)
    M, N, K = 3, 4, 5
    x, w, b, r = (rng.standard_normal(s) for s in ((M, K), (N, K), (N,), (M, N)))
    y, z, mag = linear.fwd(x, w, b, "silu", r)
    for m in range(M):
        for n in range(N):
            s = sum(x[m, k] * w[n, k] for k in range(K)) + b[n]
            assert math.isclose(z[m, n], s, rel_tol=1e-12, abs_tol=1e-14)
            assert math.isclose(y[m, n], scalar_act(s, "silu") + r[m, n], rel_tol=1e-12, abs_tol=1e-14)
            assert math.isclose(mag[m, n], sum(abs(x[m, k] * w[n, k]) for k in range(K)) + abs(b[n]), rel_tol=1e-12)
    # differences of <dy, y> in every input, with x = gelu(zx) and the layer's own silu
    zx, dy = rng.standard_normal((M, K)), rng.standard_normal((M, N))

    def loss(zx, w, b):
        return (dy * linear.fwd(linear.act(zx, "gelu_tanh"), w, b, "silu", r)[0]).sum()

    x = linear.act(zx, "gelu_tanh")
    dz = dy * linear.act_grad(linear.fwd(x, w, b, "silu", r)[1], "silu")
    dx, _, _ = linear.dgrad(dz, w, zx, "gelu_tanh", None)
    dw, _, db, _ = linear.wgrad(dz, x)
    h = 1e-6
    for g, at, arg in ((dx, zx, 0), (dw, w, 1), (db, b, 2)):
        for i in np.ndindex(*at.shape):
            args = [zx, w, b]
            hi, lo = at.copy(), at.copy()
            hi[i] += h
            lo[i] -= h
            args[arg] = hi
            up = loss(*args)
            args[arg] = lo
            assert abs((up - loss(*args)) / (2 * h) - g[i]) < 1e-7
    add = rng.standard_normal((M, K))
    assert np.allclose(linear.dgrad(dz, w, zx, "gelu_tanh", add)[0], dx + add)


def test_rows():
    rng = np.random.default_rng(1)
    T, k, H = 4, 3, 2
    inv = rng.permutation(T * k).reshape(T, k)
    inv[1, 1], inv[2, 0] = -1, T * k
    n = T * k - 3
    x, y, w, res = (rng.standard_normal(s) for s in ((T, H), (T * k, H), (T, k), (T, H)))
    y[n:] = np.nan
    got = rows.dispatch(x, inv, n, np.full((T * k, H), 5.0))
    out, mag = rows.combine(y, inv, n, w, res)
    dy, dw, _ = rows.combine_grad(x, y, inv, n, w, np.full((T * k, H), 5.0))
    seen = set()
    for t in range(T):
        s = res[t].copy()
        for j in range(k):
            at = inv[t, j]
            if not 0 <= at < n:
                assert dw[t, j] == 0
                continue
            seen.add(at)
            assert (got[at] == x[t]).all() and np.allclose(dy[at], w[t, j] * x[t])
            assert math.isclose(dw[t, j], sum(x[t] * y[at]), rel_tol=1e-12)
            s += w[t, j] * y[at]
        assert np.allclose(out[t], s) and (mag[t] >= np.abs(out[t]) - 1e-12).all()
    rest = [i for i in range(T * k) if i not in seen]
    assert (got[rest] == 5).all() and (dy[rest] == 5).all()
