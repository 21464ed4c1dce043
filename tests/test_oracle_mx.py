"""Pins of the float64 definitions in oracle/mx.py: formats by brute force, gradients by
differences."""
import numpy as np
import pytest

from oracle import mx


def test_mxfp4_nearest_value_and_scale_rule():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((64, 96)) * 2.0 ** rng.integers(-30, 30, (64, 1))).astype(np.float32).astype(np.float64)
    x[3, 32:64] = 0.0
    x[4, 5] = np.inf
    x[5, 40] = np.nan
    c, s = mx.quantize_mxfp4(x)
    v = mx.dequantize_mxfp4(c, s)
    assert s[3, 1] == 0 and s[4, 0] == 255 and s[5, 1] == 255 and np.isnan(v[4, :32]).all()
    both = np.concatenate([mx.E2M1, -mx.E2M1])
    for r in range(64):
        for b in range(3):
            if s[r, b] == 255 or (r, b) == (3, 1):
                continue
            blk = x[r, 32 * b:32 * b + 32]
            e = int(np.floor(np.log2(np.abs(blk).max()))) - 2
            assert s[r, b] == e + 127
            best = np.abs(blk[:, None] / 2.0 ** e - both[None]).min(1)
            assert (np.abs(blk - v[r, 32 * b:32 * b + 32]) / 2.0 ** e == best).all()


def test_mxfp4_ties_and_zero_signs():
    x = np.zeros((1, 32))
    x[0, :8] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]   # midpoints: to the even code
    x[0, 8:10] = [-0.25, -0.0]
    c, s = mx.quantize_mxfp4(x)
    codes = np.stack([c & 15, c >> 4], -1).reshape(-1)
    assert s[0, 0] == 127 and list(codes[:10]) == [6, 0, 2, 2, 4, 4, 6, 6, 8, 8]


def test_checkpoint_scale_is_the_smallest_that_does_not_saturate():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    h = (rng.standard_normal((32, 64)) * 2.0 ** rng.integers(-20, 20, (32, 1)))
    h[0, 0], h[1, 0], h[0, 1:32], h[1, 1:32] = 448.0, 448.5, 0.1, 0.1
    c, s = mx.e4m3_checkpoint(h)
    assert s[0, 0] == 127 and s[1, 0] == 128
    amax = np.abs(h.reshape(32, 2, 32)).max(-1)
    sc = np.exp2(s.astype(np.float64) - 127)
    assert (amax <= 448 * sc).all() and (amax > 448 * sc / 2).all()
    ref = torch.from_numpy(h / np.repeat(sc, 32, -1)).float().to(torch.float8_e4m3fn)
    assert (ref.view(torch.uint8).numpy() == c).all()
    v = mx.read_checkpoint(c, s)
    assert (np.abs(v - h) <= np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -10 * np.repeat(sc, 32, -1))).all()


def test_product_against_loops():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((5, 7)), rng.standard_normal((3, 4, 7))
    offsets, rows = np.array([0, 2, 2, 4]), np.array([4, 0, 1, 1, 2])
    out, _ = mx.product(x, w, offsets, rows, np.full((5, 4), 9.0))
    for pos, e in ((0, 0), (1, 0), (2, 2), (3, 2)):
        for n in range(4):
            assert abs(out[pos, n] - sum(x[rows[pos], i] * w[e, n, i] for i in range(7))) < 1e-12
    assert (out[4] == 9.0).all()


def test_swiglu_gradient_by_differences():
    rng = np.random.default_rng(3)
    h, da, w = rng.standard_normal((3, 8)), rng.standard_normal((3, 4)), rng.random(3)
    dh, dw = mx.swiglu_bwd(h, da, w)
    f = lambda h, w: (w[:, None] * mx.swiglu(h) * da).sum()  # noqa: E731
    eps = 1e-6
    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = eps
        assert abs((f(h + d, w) - f(h - d, w)) / (2 * eps) - dh[i]) < 1e-8
    for i in range(3):
        d = np.zeros(3)
        d[i] = eps
        assert abs((f(h, w + d) - f(h, w - d)) / (2 * eps) - dw[i]) < 1e-8


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_router_gradient_by_differences(renorm, masked):
    rng = np.random.default_rng(4)
    T, E, k = 5, 6, 2
    l = rng.standard_normal((T, E))
    if masked:
        l[:, 4] = -np.inf
    idx = np.argsort(-l, axis=1)[:, :k].copy()
    idx[0] = idx[0, 0]            # the same index twice
    idx[1, 1] = E + 3             # a dropped pair
    valid = np.array([1, 1, 0, 1, 1])
    counts, _ = mx.router_loss(l, idx, valid)
    assert counts[E] == 4 and counts[:E].sum() == 7
    dw, dloss = rng.standard_normal((T, k)), np.array([0.7, 0.3])
    g, size = mx.router_grad(l, idx, valid, counts, dw, dloss, renorm)
    assert (np.abs(g) <= size + 1e-15).all() and (g[2] == 0).all()

    def f(l):
        # the counts do not move: equal to those of l for small steps, as idx is given
        _, loss = mx.router_loss(l, idx, valid)
        return loss @ dloss + (mx.topk_weights(l, idx, renorm) * dw * valid[:, None]).sum()

    eps = 1e-6
    for i in np.ndindex(l.shape):
        if not np.isfinite(l[i]):
            assert g[i] == 0
            continue
        d = np.zeros_like(l)
        d[i] = eps
        assert abs((f(l + d) - f(l - d)) / (2 * eps) - g[i]) < 1e-7, i


def test_router_rows_and_batches_of_nothing():
    l = np.full((2, 4), -np.inf)
    idx = np.zeros((2, 1), np.int64)
    counts, loss = mx.router_loss(l, idx)
    assert (loss == 0).all() and list(counts) == [2, 0, 0, 0, 2]
    counts, loss = mx.router_loss(l, idx, np.zeros(2))
    assert (loss == 0).all() and (counts == 0).all()
