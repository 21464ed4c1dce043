"""MXFP4 quantization, the experts' product and its input gradient, SwiGLU with an 8-bit
checkpoint, and the router's losses and gradient, in float64.

Test infrastructure (see the package docstring).  MXFP4 is the OCP microscaling format:
blocks of 32, E8M0 scales (a byte c stands for 2^(c - 127), 255 for NaN), E2M1 elements.
Readings: a zero block has scale code 0; a block with an infinity or NaN has code 255 and
element codes 0; the scale exponent is clamped at -127.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the non-negative E4M3FN values by code: 8 subnormals, then 15 binades, without the NaN
E4M3 = np.array([m / 512.0 for m in range(8)] +
                [(1 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1])
BLOCK = 32


def _code_of(v, grid):
    """Place of the nearest grid value to v >= 0, ties to the even place, saturating."""
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def _blocks(x):
    x = np.asarray(x, dtype=np.float64)
    return x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)


def quantize_mxfp4(x):
    """x [..., cols] (bf16 values) -> codes uint8 [..., cols/2], scales uint8 [..., cols/32]."""
    b = _blocks(x)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    s = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127)
    s = np.maximum(s, -127)
    c = _code_of(np.abs(b) / np.exp2(s.astype(np.float64))[..., None], E2M1).astype(np.uint8)
    c |= (np.signbit(b) & ~bad[..., None]).astype(np.uint8) << 3
    c = c.reshape(*c.shape[:-2], c.shape[-2] * BLOCK)
    return c[..., 0::2] | (c[..., 1::2] << 4), np.where(bad, 255, s + 127).astype(np.uint8)


def dequantize_mxfp4(codes, scales):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    sc = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (_blocks(v) * sc[..., None]).reshape(v.shape)


def product(x, w, offsets, rows, out):
    """out[pos] = x[rows[pos]] w[e]^T over each expert's positions (others left); also the
    sum of the products' magnitudes, for error bounds."""
    mag = np.zeros_like(out)
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            out[a:b] = x[rows[a:b]] @ w[e].T
            mag[a:b] = np.abs(x[rows[a:b]]) @ np.abs(w[e]).T
    return out, mag


def e4m3_checkpoint(h):
    """h [..., cols] -> E4M3 bytes, E8M0 codes: the smallest 2^s with max|h| <= 448 2^s."""
    b = _blocks(h)
    bad = ~np.isfinite(b).all(-1)
    amax = np.abs(np.where(bad[..., None], 0.0, b)).max(-1)
    m, e = np.frexp(amax)
    s = np.where(amax > 0, np.where(m <= 0.875, e - 9, e - 8), -127)
    s = np.maximum(s, -127)
    c = _code_of(np.abs(np.where(bad[..., None], 0.0, b)) / np.exp2(s.astype(np.float64))[..., None], E4M3).astype(np.uint8)
    c |= np.signbit(b).astype(np.uint8) << 7
    return c.reshape(h.shape), np.where(bad, 255, s + 127).astype(np.uint8)


def read_checkpoint(c, s):
    sc = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    v = np.where(c & 128, -1.0, 1.0) * E4M3[np.minimum(c & 127, 126)]
    return (_blocks(v) * sc[..., None]).reshape(c.shape)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def swiglu(h):
    g, u = np.split(h, 2, axis=-1)
    return g * sigmoid(g) * u


def swiglu_bwd(h, da, w):
    """h, da [R, ...], w [R] -> dh, and per row sum da silu(g) u."""
    g, u = np.split(h, 2, axis=-1)
    s = sigmoid(g)
    d = w[:, None] * da
    return np.concatenate([d * u * s * (1 + g * (1 - s)), d * g * s], -1), (da * g * s * u).sum(-1)


def softmax(l):
    m = l.max(-1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    ex = np.exp(l - m)
    s = ex.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(s[..., 0] > 0, m[..., 0] + np.log(s[..., 0]), 0.0)
    return np.divide(ex, s, out=np.zeros_like(ex), where=s > 0), lse


def router_loss(l, idx, valid=None):
    """-> counts [E + 1], (balance loss, z-loss)."""
    T, E = l.shape
    keep = np.ones(T, bool) if valid is None else valid != 0
    l, idx = l[keep].astype(np.float64), idx[keep]
    n, k = idx.shape
    inside = idx[(idx >= 0) & (idx < E)]
    counts = np.bincount(inside, minlength=E)
    if n == 0:
        return np.append(counts, 0), np.zeros(2)
    p, lse = softmax(l)
    return np.append(counts, n), np.array([E * (counts / (n * k) * p.mean(0)).sum(), (lse ** 2).mean()])


def topk_weights(l, idx, renorm):
    """softmax probabilities at the given indices (0 where outside [0, E)), renormalised if asked."""
    p, _ = softmax(l.astype(np.float64))
    ok = (idx >= 0) & (idx < l.shape[1])
    q = np.where(ok, np.take_along_axis(p, np.where(ok, idx, 0), 1), 0.0)
    if renorm:
        s = q.sum(1, keepdims=True)
        q = np.divide(q, s, out=np.zeros_like(q), where=s > 0)
    return q


def router_grad(l, idx, valid, counts, dw, dloss, renorm):
    """Gradient of dloss . losses + sum dw topk_w in the logits; and, for error bounds, the
    sum of the magnitudes of its terms."""
    T, E = l.shape
    k = idx.shape[1]
    keep = np.ones(T, bool) if valid is None else valid != 0
    l = np.where(keep[:, None], l.astype(np.float64), 0.0)
    n = counts[E]
    p, lse = softmax(l)
    up = np.zeros((T, E))
    if n:
        up += dloss[0] * E * counts[:E] / (n * k) / n
    size = np.abs(up)
    ok = (idx >= 0) & (idx < E)
    d = np.where(ok & keep[:, None], np.nan_to_num(dw.astype(np.float64)), 0.0)
    q = np.where(ok, np.take_along_axis(p, np.where(ok, idx, 0), 1), 0.0)
    if renorm:
        s = q.sum(1, keepdims=True)
        r = np.divide(1.0, s, out=np.zeros_like(s), where=s > 0)
        dq = (d - (q * d).sum(1, keepdims=True) * r) * r
        mag = (np.abs(d) + (q * np.abs(d)).sum(1, keepdims=True) * r) * r
    else:
        dq, mag = d, np.abs(d)
    t = np.repeat(np.arange(T), k).reshape(T, k)
    np.add.at(up, (t[ok], idx[ok]), dq[ok])
    np.add.at(size, (t[ok], idx[ok]), mag[ok])
    gz = 2 * dloss[1] / n if n else 0.0
    g = p * (up - (p * up).sum(1, keepdims=True) + gz * lse[:, None])
    size = p * (size + (p * size).sum(1, keepdims=True) + np.abs(gz * lse[:, None]))
    return np.where(keep[:, None], g, 0.0), np.where(keep[:, None], size, 0.0)
