"""GPU parity of the MXFP4 quantizer, the experts' product and its input gradient, SwiGLU
with the 8-bit checkpoint, and the router's losses and gradient, against oracle/mx.py.

Tolerances, per element (u = 2^-24, bf16 rounds to within 2^-8 of a value):
* products: the 4-bit (or bf16) products are exact in FP32 and at most K additions are off
  by one unit in the last place (2^-23) of a partial sum no larger than S = sum |x w| each:
  2^-8 |ref| + K 2^-23 S.
* SwiGLU: sigmoid's error is that of e^-g, (|g| + 8) u with its reciprocal; a product of it
  adds a few u: 2^-8 |ref| + (|g| + 16) 2^-23 |terms|.  Beyond |g| = 88 e^-g overflows
  and silu is 0 for |g| e^-88 < 1e-35.
* router: no path from a logit to an output has more than 64 FP32 roundings: 2^-18 of the
  sum of the magnitudes of the terms; the losses, sums of positive terms: 2^-18 relative.
"""
import numpy as np
import pytest

from oracle import mx
from tests.gpu_util import gpu, log

pytestmark = pytest.mark.gpu


def _bqm():
    import bit_quantized_moe_amd as bqm
    return bqm


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(dtype) if dtype is not None else t).to(gpu())


def bf16(a):
    """float -> the nearest bf16 values, as float64."""
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def dev_bf16(a):
    import torch
    return dev(np.asarray(a, dtype=np.float32), torch.bfloat16)


def host(t):
    t = t.detach()
    return (t.double() if t.is_floating_point() else t).cpu().numpy()


def within(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]}, {tol[bad][0]} allowed")


# ---------------------------------------------------------------------------
# MXFP4
# ---------------------------------------------------------------------------
def quantize(x):
    """x float64 of bf16 values [n, rows, cols] -> device QTensor."""
    bqm = _bqm()
    return bqm.quantize_stack(dev_bf16(x), "mxfp4")


def check_quant(x):
    q = quantize(x)
    c, s = mx.quantize_mxfp4(x)
    assert (host(q.scales) == s).all()
    assert (host(q.codes) == c).all()
    return q, c, s


@pytest.mark.parametrize("shape", [(1, 1, 32), (3, 5, 96), (2, 37, 480), (1, 130, 2080), (5, 1, 1024)])
def test_mxfp4_bit_exact(shape):
    log(f"mxfp4 {shape}")
    rng = np.random.default_rng(shape[1])
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-40, 40, shape[:2] + (1,)))
    x[rng.random(shape) < 0.05] = 0.0
    x[..., :32] *= rng.random(shape[:2] + (1,)) < 0.7
    q, c, s = check_quant(bf16(x))
    import torch
    y = torch.empty(shape, dtype=torch.bfloat16, device=gpu())
    _bqm().bqm_dequantize(q, y)
    assert (host(y) == mx.dequantize_mxfp4(c, s)).all()


def test_mxfp4_every_block_maximum():
    """All 32768 bf16 magnitudes as a block's maximum (zero, subnormals, infinity, NaN), over
    elements that fall on every E2M1 midpoint of that block's scale."""
    log("mxfp4 block maxima")
    mags = np.arange(1 << 15, dtype=np.uint32)
    with np.errstate(invalid="ignore"):
        top = (mags << 16).view(np.float32).astype(np.float64)
        unit = np.where(np.isfinite(top) & (top > 0), np.exp2(np.maximum(np.frexp(np.where(np.isfinite(top), top, 1))[1] - 3, -127).astype(np.float64)), 1.0)
    pat = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 0.2490234375, 0.251953125, 1.5, 2.0, 3.0, 0.5, 0.0, 1.0, 4.0] * 2)
    pat[15:] *= -1
    x = np.zeros((1, 1 << 15, 32))
    x[0, :, :30] = np.where(pat[None] * unit[:, None] <= top[:, None], pat[None] * unit[:, None], 0.0)
    x[0, :, :30] = np.maximum(x[0, :, :30], -np.where(np.isfinite(top), top, 4.0)[:, None])
    x = bf16(x)
    x[0, :, 30] = top
    x[0, 1::2, 30] *= -1
    x[0, :, 31] = -0.0
    check_quant(x)


def test_mxfp4_decodes_every_code_and_scale():
    import torch
    bqm = _bqm()
    q = bqm.alloc_qtensor(bqm.FMT_MXFP4, 1, 256, 32)
    q.codes.copy_(dev(np.tile(np.arange(16, dtype=np.uint8) * 16 + np.arange(15, -1, -1, dtype=np.uint8), (1, 256, 1))))
    q.scales.copy_(dev(np.arange(256, dtype=np.uint8).reshape(1, 256, 1)))
    y = torch.empty((1, 256, 32), dtype=torch.bfloat16, device=gpu())
    bqm.bqm_dequantize(q, y)
    ref = mx.dequantize_mxfp4(host(q.codes), host(q.scales))
    ref = np.where(np.abs(ref) >= 2.0 ** 128, np.copysign(np.inf, ref), ref)   # 4 and 6 times 2^126, 2^127
    got = host(y)
    assert np.array_equal(got, ref, equal_nan=True) and (np.signbit(got) == np.signbit(ref))[~np.isnan(ref)].all()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def routed(rng, T, E, k, kind):
    """idx [T, k] and its permutation by the library; kind: even | zipf | one (all on one
    expert) | dropped (some indices outside [0, E))."""
    import torch
    bqm = _bqm()
    score = rng.random((T, E))
    if kind == "zipf":
        score -= np.log(1 + rng.permutation(E))
    if kind == "one":
        score[:, E - 1] += 10
    idx = np.argsort(-score, axis=1)[:, :k].astype(np.int32)
    if kind == "dropped":
        idx[rng.random((T, k)) < 0.3] = -1
        idx[rng.random((T, k)) < 0.1] = E + 7
    R = T * k
    perm, inv = (torch.empty(R, dtype=torch.int32, device=gpu()) for _ in range(2))
    offsets = torch.empty(E + 1, dtype=torch.int32, device=gpu())
    ws = torch.empty(max(16, bqm.bqm_permute_workspace_size(T, E, k)), dtype=torch.uint8, device=gpu())
    bqm.bqm_permute(dev(idx), T, E, k, perm, inv, offsets, ws)
    return idx, perm, inv, offsets


SHAPES = [  # E, T, k, N, K, kind
    (1, 1, 1, 32, 32, "even"),
    (8, 1, 2, 64, 96, "even"),
    (8, 3, 2, 288, 512, "even"),
    (60, 9, 4, 160, 2080, "zipf"),
    (16, 33, 2, 256, 256, "dropped"),
    (5, 70, 3, 96, 736, "zipf"),
    (4, 200, 2, 544, 1024, "one"),
    (3, 700, 1, 320, 1536, "even"),
    (7, 259, 4, 1056, 160, "dropped"),
    (128, 64, 8, 128, 768, "even"),
    (1024, 40, 2, 64, 64, "even"),
    (4, 60, 2, 288, 384, "zipf"),
    (5, 110, 2, 1120, 256, "dropped"),
    (2, 150, 1, 64, 128, "even"),
]


def product_case(E, T, k, N, K, kind, gather, seed=0):
    rng = np.random.default_rng([E, T, k, N, K, gather, seed])
    idx, perm, inv, offsets = routed(rng, T, E, k, kind)
    R = T * k
    w = bf16(rng.standard_normal((E, N, K)) * 0.02 * np.exp2(rng.integers(-3, 4, (E, N, 1))))
    rows = host(perm) // k if gather else np.arange(R)
    return rng, R, w, rows, perm if gather else None, offsets, host(offsets)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,k,N,K,kind", SHAPES)
def test_gemm_against_oracle(E, T, k, N, K, kind, gather):
    import torch
    log(f"mxfp4_gemm E={E} T={T} k={k} N={N} K={K} {kind} gather={gather}")
    bqm = _bqm()
    rng, R, w, rows, perm, offsets, off = product_case(E, T, k, N, K, kind, gather)
    x = bf16(rng.standard_normal((T if gather else R, K)) * np.exp2(rng.integers(-2, 3, (T if gather else R, 1))))
    wq, xq = quantize(w), quantize(x[None])
    mark = 7.0
    y = torch.full((R, N), mark, dtype=torch.bfloat16, device=gpu())
    bqm.bqm_mxfp4_gemm(xq, wq, offsets, perm, k, y)
    ref, mag = mx.product(mx.dequantize_mxfp4(*mx.quantize_mxfp4(x)), mx.dequantize_mxfp4(*mx.quantize_mxfp4(w)), off,
                          rows, np.full((R, N), mark))
    within(host(y), ref, 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag, "y")
    assert (host(y)[off[E]:] == mark).all()
    y2 = torch.full_like(y, mark)
    bqm.bqm_mxfp4_gemm(xq, wq, offsets, perm, k, y2)
    assert torch.equal(y, y2), "two calls differ"


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,k,N,K,kind", SHAPES)
def test_dgrad_against_oracle(E, T, k, N, K, kind, gather):
    import torch
    log(f"mxfp4_dgrad E={E} T={T} k={k} N={N} K={K} {kind} gather={gather}")
    bqm = _bqm()
    rng, R, w, rows, perm, offsets, off = product_case(E, T, k, N, K, kind, gather)
    dy = bf16(rng.standard_normal((T if gather else R, N)))
    mark = 7.0
    dx = torch.full((R, K), mark, dtype=torch.bfloat16, device=gpu())
    wq = quantize(w)
    bqm.bqm_mxfp4_dgrad(wq, dev_bf16(dy), offsets, perm, k, dx)
    wv = mx.dequantize_mxfp4(*mx.quantize_mxfp4(w))
    ref, mag = mx.product(dy, np.ascontiguousarray(wv.transpose(0, 2, 1)), off, rows, np.full((R, K), mark))
    within(host(dx), ref, 2.0 ** -8 * np.abs(ref) + N * 2.0 ** -23 * mag, "dx")
    assert (host(dx)[off[E]:] == mark).all()


# Rows of the experts: row tiles of 256 rows in every number that the largest tile's kernels
# walk in another way (1, 2, 4 and 5 in one group; 6 = 3 + 3, 7 = 4 + 3, 9 = 5 + 4,
# 13 = 5 + 5 + 3 in groups), whole or ending one row into a tile, and an expert without rows.
WALK = [1025, 0, 1536, 1, 1537, 2049, 300, 3200, 1000]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("kind,N,K", [("gemm", 1056, 256), ("gemm", 544, 736), ("gemm", 800, 224),
                                      ("dgrad", 96, 1152), ("dgrad", 64, 640), ("dgrad", 160, 800), ("dgrad", 32, 544)])
def test_walk_of_many_row_and_column_tiles(kind, N, K, gather):
    """Experts of many row tiles over several column tiles, the last of them partly filled;
    every row of an expert is written, no other is.  With the copies of whole 128-byte steps
    (product 256 and 736, gradient 1152 and 640) and without."""
    import torch
    log(f"walk {kind} N={N} K={K} gather={gather}")
    bqm = _bqm()
    rng = np.random.default_rng([N, K, gather])
    off = np.concatenate([[0], np.cumsum(WALK)]).astype(np.int32)
    E, k = len(WALK), 2
    R = int(off[E]) + 38
    assert R % k == 0 and R >= 128 * E
    perm = rng.permutation(R).astype(np.int32) if gather else None
    rows, src = (perm // k, R // k) if gather else (np.arange(R), R)
    w = bf16(rng.standard_normal((E, N, K)) * 0.05)
    wq, wv = quantize(w), mx.dequantize_mxfp4(*mx.quantize_mxfp4(w))
    x = bf16(rng.standard_normal((src, K if kind == "gemm" else N)))
    mark = 7.0
    out = torch.full((R, N if kind == "gemm" else K), mark, dtype=torch.bfloat16, device=gpu())
    d_perm = dev(perm) if gather else None
    if kind == "gemm":
        bqm.bqm_mxfp4_gemm(quantize(x[None]), wq, dev(off), d_perm, k, out)
        x = mx.dequantize_mxfp4(*mx.quantize_mxfp4(x))
    else:
        bqm.bqm_mxfp4_dgrad(wq, dev_bf16(x), dev(off), d_perm, k, out)
        wv = np.ascontiguousarray(wv.transpose(0, 2, 1))
    ref, mag = mx.product(x, wv, off, rows, np.full(out.shape, mark))
    within(host(out), ref, 2.0 ** -8 * np.abs(ref) + x.shape[1] * 2.0 ** -23 * mag, "out")
    assert (host(out)[off[E]:] == mark).all()


def test_products_with_extreme_scales_and_nan_blocks():
    """Rows and columns over the whole range of scales; a NaN block reaches its own row (or
    column) only, and the experts without rows are not read."""
    import torch
    log("mxfp4 products, extreme scales")
    bqm = _bqm()
    rng = np.random.default_rng(9)
    E, T, N, K = 3, 6, 64, 288
    w = bf16(rng.standard_normal((E, N, K)) * np.exp2(rng.integers(-100, 100, (E, N, 1)).astype(np.float64)))
    x = bf16(rng.standard_normal((T, K)) * np.exp2(rng.integers(-20, 20, (T, 1)).astype(np.float64)))
    x[2, 40] = np.inf
    w[0, 5, 287] = np.nan
    w[1] = np.nan                                  # no rows
    off = np.array([0, 4, 4, 6], dtype=np.int32)
    y = torch.empty((T, N), dtype=torch.bfloat16, device=gpu())
    bqm.bqm_mxfp4_gemm(quantize(x[None]), quantize(w), dev(off), None, 1, y)
    ref, mag = mx.product(mx.dequantize_mxfp4(*mx.quantize_mxfp4(x)), mx.dequantize_mxfp4(*mx.quantize_mxfp4(w)), off,
                          np.arange(T), np.zeros((T, N)))
    got = host(y)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.isnan(ref).sum() == N + 3
    ok = ~np.isnan(ref)
    within(got[ok], ref[ok], (2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag)[ok], "y")
    dy = bf16(rng.standard_normal((T, N)))
    w[0, 5, 287] = 1.0
    dx = torch.empty((T, K), dtype=torch.bfloat16, device=gpu())
    bqm.bqm_mxfp4_dgrad(quantize(w), dev_bf16(dy), dev(off), None, 1, dx)
    wv = mx.dequantize_mxfp4(*mx.quantize_mxfp4(w))
    ref, mag = mx.product(dy, np.ascontiguousarray(wv.transpose(0, 2, 1)), off, np.arange(T), np.zeros((T, K)))
    within(host(dx), ref, 2.0 ** -8 * np.abs(ref) + N * 2.0 ** -23 * mag, "dx")


@pytest.mark.parametrize("K", [256, 96])
def test_products_with_scales_past_bf16(K):
    """A weight row with the two largest scale codes, whose values reach 6 2^127: the product
    multiplies the values, the gradient what the dequantizer gives (infinity from 2^128 on)."""
    import torch
    log(f"mxfp4 products, scale codes 253 and 254, K={K}")
    bqm = _bqm()
    rng = np.random.default_rng(K)
    N = 64
    w = quantize(bf16(rng.standard_normal((1, N, K))))
    w.codes[0, 3].copy_(dev(rng.integers(0, 256, K // 2).astype(np.uint8)))
    w.scales[0, 3].copy_(dev(np.where(np.arange(K // 32) % 2, 254, 253).astype(np.uint8)))
    x = bf16(rng.standard_normal((5, K)) * 2.0 ** -40)
    off = dev(np.array([0, 5], np.int32))
    y = torch.empty((5, N), dtype=torch.bfloat16, device=gpu())
    bqm.bqm_mxfp4_gemm(quantize(x[None]), w, off, None, 1, y)
    ref, mag = mx.product(mx.dequantize_mxfp4(*mx.quantize_mxfp4(x)), mx.dequantize_mxfp4(host(w.codes), host(w.scales)),
                          [0, 5], np.arange(5), np.zeros((5, N)))
    within(host(y), ref, 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag, "y")
    dy = np.zeros((5, N))
    dy[:, 3] = [1, -1, 0.5, 2.0 ** -9, -2.0]
    dx, dq = (torch.empty(s, dtype=torch.bfloat16, device=gpu()) for s in ((5, K), (1, N, K)))
    bqm.bqm_mxfp4_dgrad(w, dev_bf16(dy), off, None, 1, dx)
    bqm.bqm_dequantize(w, dq)
    wv = host(dq)[0, 3]
    assert np.isinf(wv).any() and not np.isinf(wv).all()
    with np.errstate(over="ignore"):        # -2 times 2^127 and more is past bf16 as well
        want = bf16(dy[:, 3:4] * wv)
    assert np.array_equal(host(dx), want)


@pytest.mark.parametrize("kind,N,K", [("gemm", 96, 256), ("gemm", 160, 96), ("dgrad", 64, 256), ("dgrad", 96, 160)])
@pytest.mark.parametrize("R", [64, 1500])
def test_offsets_and_rows_out_of_range_are_clamped(kind, N, K, R):
    """Offsets below 0, past R and falling, and source rows of no token: a result is the row's
    expert's product of the clamped source row, that of any of its experts where offsets that
    fall give it to several, and what it was where they give it to none."""
    import torch
    log(f"clamped {kind} N={N} K={K} R={R}")
    bqm = _bqm()
    rng = np.random.default_rng([N, K, R])
    k = 2
    off = np.array([5, R // 4, R // 4 + 3, R // 8, R // 2, R // 2, 3 * R // 4, R // 2 + 5, (1 << 31) - 1, -7, 3,
                    -(1 << 31)], np.int32)
    E = len(off) - 1
    perm = rng.integers(0, R, R).astype(np.int32)
    wild = rng.random(R) < 0.2
    perm[wild] = np.array([-1, -9, R, R + 5, (1 << 31) - 1, -(1 << 31)])[rng.integers(0, 6, wild.sum())]
    src = R // k
    rows = np.clip(np.trunc(perm / k).astype(np.int64), 0, src - 1)
    w = bf16(rng.standard_normal((E, N, K)) * 0.05)
    wq, wv = quantize(w), mx.dequantize_mxfp4(*mx.quantize_mxfp4(w))
    x = bf16(rng.standard_normal((src, K if kind == "gemm" else N)))
    mark = 7.0
    # rows of the mark on both sides of the output, too
    whole = torch.full((R + 512, N if kind == "gemm" else K), mark, dtype=torch.bfloat16, device=gpu())
    out = whole[256:256 + R]
    if kind == "gemm":
        bqm.bqm_mxfp4_gemm(quantize(x[None]), wq, dev(off), dev(perm), k, out)
        x = mx.dequantize_mxfp4(*mx.quantize_mxfp4(x))
    else:
        bqm.bqm_mxfp4_dgrad(wq, dev_bf16(x), dev(off), dev(perm), k, out)
        wv = np.ascontiguousarray(wv.transpose(0, 2, 1))
    got, at = host(whole), np.clip(off.astype(np.int64), 0, R)
    assert (got[:256] == mark).all() and (got[256 + R:] == mark).all()
    got, owners = got[256:256 + R], np.zeros(R, int)
    found = np.zeros(got.shape, bool)
    for e in range(E):
        a, b = at[e], at[e + 1]
        if b <= a:
            continue
        ref, mag = x[rows[a:b]] @ wv[e].T, np.abs(x[rows[a:b]]) @ np.abs(wv[e]).T
        found[a:b] |= np.abs(got[a:b] - ref) <= 2.0 ** -8 * np.abs(ref) + x.shape[1] * 2.0 ** -23 * mag
        owners[a:b] += 1
    assert (owners == 0).any() and (owners == 1).any() and (owners > 1).any()
    assert found[owners > 0].all() and (got[owners == 0] == mark).all()


def test_products_past_four_gigabytes_of_weights():
    import torch
    log("mxfp4 products, expert stack over 4 GiB")
    bqm = _bqm()
    E, N, K, k = 600, 2048, 8192, 1
    g = torch.Generator(device=gpu()).manual_seed(1)
    q = bqm.alloc_qtensor(bqm.FMT_MXFP4, E, N, K)
    assert q.codes.numel() > 1 << 32
    q.codes.zero_()
    q.scales.fill_(127)
    hit = (3, 530, 599)
    for e in hit:
        q.codes[e].copy_(torch.randint(0, 256, (N, K // 2), generator=g, device=gpu(), dtype=torch.uint8))
    rng = np.random.default_rng(5)
    x = bf16(rng.standard_normal((3, K)))
    off = np.zeros(E + 1, dtype=np.int32)
    for i, e in enumerate(hit):
        off[e + 1:] = i + 1
    y = torch.empty((3, N), dtype=torch.bfloat16, device=gpu())
    dx = torch.empty((3, K), dtype=torch.bfloat16, device=gpu())
    dy = bf16(rng.standard_normal((3, N)))
    bqm.bqm_mxfp4_gemm(quantize(x[None]), q, dev(off), None, 1, y)
    bqm.bqm_mxfp4_dgrad(q, dev_bf16(dy), dev(off), None, 1, dx)
    xv = mx.dequantize_mxfp4(*mx.quantize_mxfp4(x))
    for i, e in enumerate(hit):
        w = mx.dequantize_mxfp4(host(q.codes[e]), host(q.scales[e]))
        ref, mag = xv[i] @ w.T, np.abs(xv[i]) @ np.abs(w).T
        within(host(y[i]), ref, 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag, f"y {e}")
        ref, mag = dy[i] @ w, np.abs(dy[i]) @ np.abs(w)
        within(host(dx[i]), ref, 2.0 ** -8 * np.abs(ref) + N * 2.0 ** -23 * mag, f"dx {e}")


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("gib", [3.5, 4.5])
def test_products_of_large_activations(gib, gather):
    """Source rows past 2 and 4 GiB, gathered in a random order or as they lie; a sample of
    the results against the oracle."""
    import torch
    log(f"mxfp4 products, activations of {gib} GiB, gather={gather}")
    bqm = _bqm()
    gen = torch.Generator(device=gpu()).manual_seed(3)
    K, N = 4096, 32
    R = int(gib * 2 ** 30) // (K // 2)
    x = bqm.alloc_qtensor(bqm.FMT_MXFP4, 1, R, K)
    x.codes.random_(0, 256, generator=gen)
    x.scales.random_(120, 130, generator=gen)
    w = quantize(bf16(np.random.default_rng(1).standard_normal((2, N, K))))
    perm = torch.randperm(R, generator=gen, device=gpu()).int() if gather else None
    off = np.array([0, R // 3, R], np.int32)
    y = torch.empty((R, N), dtype=torch.bfloat16, device=gpu())
    bqm.bqm_mxfp4_gemm(x, w, dev(off), perm, 1, y)
    pos = np.unique(np.concatenate([[0, R // 3 - 1, R // 3, R - 1], np.random.default_rng(2).integers(0, R, 200)]))
    rows = host(perm[dev(pos)]) if gather else pos
    e = (pos >= off[1]).astype(int)
    wv = mx.dequantize_mxfp4(host(w.codes), host(w.scales))
    xv = mx.dequantize_mxfp4(host(x.codes[0, dev(rows)]), host(x.scales[0, dev(rows)]))
    ref, mag = (np.stack([f(wv[e[i]]) @ f(xv[i]) for i in range(len(pos))]) for f in (np.asarray, np.abs))
    within(host(y[dev(pos)]), ref, 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag, "y")
    del x, y
    K, N = 128, 4096
    R = int(gib * 2 ** 30) // (2 * N)
    dy = torch.randn((R, N), generator=gen, device=gpu(), dtype=torch.bfloat16)
    w = quantize(bf16(np.random.default_rng(1).standard_normal((2, N, K))))
    perm = torch.randperm(R, generator=gen, device=gpu()).int() if gather else None
    off = np.array([0, R // 3, R], np.int32)
    dx = torch.empty((R, K), dtype=torch.bfloat16, device=gpu())
    bqm.bqm_mxfp4_dgrad(w, dy, dev(off), perm, 1, dx)
    pos = np.unique(np.concatenate([[0, R // 3 - 1, R // 3, R - 1], np.random.default_rng(2).integers(0, R, 200)]))
    rows = host(perm[dev(pos)]) if gather else pos
    e = (pos >= off[1]).astype(int)
    wv = mx.dequantize_mxfp4(host(w.codes), host(w.scales))
    dv = host(dy[dev(rows)])
    ref, mag = (np.stack([f(dv[i]) @ f(wv[e[i]]) for i in range(len(pos))]) for f in (np.asarray, np.abs))
    within(host(dx[dev(pos)]), ref, 2.0 ** -8 * np.abs(ref) + N * 2.0 ** -23 * mag, "dx")


def test_dgrad_is_the_products_difference():
    """The product is linear, so its differences along the unit vectors are its derivative:
    rows of one 1 give W's columns, and the gradient of one output W's rows, both exactly."""
    import torch
    log("dgrad against the product's differences")
    bqm = _bqm()
    rng = np.random.default_rng(8)
    E, N, K = 3, 160, 96
    w = quantize(bf16(rng.standard_normal((E, N, K)) * np.exp2(rng.integers(-9, 9, (E, N, 1)).astype(np.float64))))
    y = torch.empty((E * K, N), dtype=torch.bfloat16, device=gpu())
    dx = torch.empty((E * N, K), dtype=torch.bfloat16, device=gpu())
    bqm.bqm_mxfp4_gemm(quantize(np.tile(np.eye(K), (E, 1))[None]), w, dev(np.arange(E + 1, dtype=np.int32) * K), None,
                       1, y)
    bqm.bqm_mxfp4_dgrad(w, dev_bf16(np.tile(np.eye(N), (E, 1))), dev(np.arange(E + 1, dtype=np.int32) * N), None, 1,
                        dx)
    assert torch.equal(y.reshape(E, K, N).transpose(1, 2), dx.reshape(E, N, K))


# ---------------------------------------------------------------------------
# SwiGLU with the 8-bit checkpoint
# ---------------------------------------------------------------------------
def swiglu_buffers(R, I):
    import torch
    e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=gpu())  # noqa: E731
    return (e(R, 2 * I, dtype=torch.uint8), e(R, 2 * I // 32, dtype=torch.uint8), e(R, I), e(R, 2 * I))


def check_swiglu(h, da, w, perm, live, h8, s8, a, dh, dw):
    R, I = da.shape
    c, s = mx.e4m3_checkpoint(h)
    fin = s[:live] != 255
    assert (host(s8)[:live] == s[:live]).all()
    whole = np.repeat(fin, 32, -1)
    assert (host(h8)[:live][whole] == c[:live][whole]).all()
    g, u = np.split(h[:live], 2, -1)
    with np.errstate(invalid="ignore"):
        ref = mx.swiglu(h[:live])
        ok = np.isfinite(ref)
        tol = 2.0 ** -8 * np.abs(ref) + (np.abs(g) + 16) * 2.0 ** -23 * np.abs(ref) + 1e-35 * np.abs(u)
    within(host(a)[:live][ok], ref[ok], tol[ok], "a")
    v = mx.read_checkpoint(c, s)[:live]
    wr = w[perm[:live]]
    ref, dot = mx.swiglu_bwd(v, da[:live], wr)
    g, u = np.split(v, 2, -1)
    sg = mx.sigmoid(g)
    d = np.abs(wr[:, None] * da[:live])
    terms = np.concatenate([d * np.abs(u) * sg * (1 + np.abs(g) * (1 - sg)), d * np.abs(g) * sg], -1)
    eps = (np.abs(np.concatenate([g, g], -1)) + 16) * 2.0 ** -23
    small = 1e-35 * np.concatenate([d * np.abs(u), d], -1) * (1 + np.abs(np.concatenate([g, g], -1)))
    ok = np.isfinite(ref)
    within(host(dh)[:live][ok], ref[ok], (2.0 ** -8 * np.abs(ref) + eps * terms + small)[ok], "dh")
    assert np.array_equal(np.isnan(host(dh)[:live]), np.isnan(ref))
    t = np.abs(da[:live]) * np.abs(g) * sg * np.abs(u)
    tol = ((np.abs(g) + 16) * 2.0 ** -23 * t).sum(-1) + I * 2.0 ** -24 * t.sum(-1) + 1e-35 * np.abs(da[:live] * u).sum(-1)
    ok = np.isfinite(dot)
    within(host(dw).reshape(-1)[perm[:live]][ok], dot[ok], tol[ok], "dtopk_w")
    assert (host(dw).reshape(-1)[perm[live:]] == 0).all()


@pytest.mark.parametrize("R,I,live", [(1, 32, 1), (3, 96, 3), (65, 768, 65), (9, 2048, 9), (130, 160, 77), (40, 64, 0),
                                      (257, 1056, 256), (2, 8192, 2)])
def test_swiglu_checkpoint(R, I, live):
    import torch
    log(f"swiglu R={R} I={I} live={live}")
    bqm = _bqm()
    rng = np.random.default_rng([R, I])
    h = bf16(rng.standard_normal((R, 2 * I)) * np.exp2(rng.integers(-12, 5, (R, 1))))
    h[0, :4] = [120.0, -120.0, 0.0, -0.0]
    if live > 50:
        h[5, 7] = np.inf
        h[6, I + 9] = np.nan
        h[7, :32] = 0.0
    da, w = bf16(rng.standard_normal((R, I))), rng.random(R).astype(np.float32)
    perm = rng.permutation(R).astype(np.int32)
    h8, s8, a, dh = swiglu_buffers(R, I)
    a.fill_(3.0)
    dh.fill_(3.0)
    h8.fill_(9)
    s8.fill_(9)
    dw = torch.full((R,), 5.0, device=gpu())
    n = dev(np.array([live], np.int32)) if live < R else None
    aq = bqm.alloc_qtensor(bqm.FMT_MXFP4, 1, R, I)
    aq.codes.fill_(9)
    bqm.bqm_swiglu_ckpt_fwd(dev_bf16(h), h8, s8, a=a, aq=aq, n_rows=n)
    bqm.bqm_swiglu_ckpt_bwd(h8, s8, dev_bf16(da), dev(perm), dev(w), dh, dw, n_rows=n)
    check_swiglu(h, da, w.astype(np.float64), perm, live, h8, s8, a, dh, dw)
    # a in MXFP4 is what the quantizer makes of the bf16 a; either output may be left out
    c, s = mx.quantize_mxfp4(host(a)[:live])
    assert (host(aq.codes)[0, :live] == c).all() and (host(aq.scales)[0, :live] == s).all()
    assert (host(aq.codes)[0, live:] == 9).all() and (host(h8)[live:] == 9).all() and (host(s8)[live:] == 9).all()
    assert (host(a)[live:] == 3).all() and (host(dh)[live:] == 3).all()
    aq2, b8, bs = bqm.alloc_qtensor(bqm.FMT_MXFP4, 1, R, I), h8.clone(), s8.clone()
    aq2.codes.fill_(9)
    bqm.bqm_swiglu_ckpt_fwd(dev_bf16(h), b8, bs, aq=aq2, n_rows=n)
    assert torch.equal(aq2.codes, aq.codes) and torch.equal(b8, h8) and torch.equal(bs, s8)


def test_swiglu_without_perm_weights_or_their_gradient():
    import torch
    log("swiglu, optional arguments left out")
    bqm = _bqm()
    rng = np.random.default_rng(4)
    R, I = 37, 320
    h, da = bf16(rng.standard_normal((R, 2 * I))), bf16(rng.standard_normal((R, I)))
    h8, s8, a, dh = swiglu_buffers(R, I)
    dw, dh2 = torch.empty(R, device=gpu()), torch.empty_like(dh)
    bqm.bqm_swiglu_ckpt_fwd(dev_bf16(h), h8, s8, a=a)
    bqm.bqm_swiglu_ckpt_bwd(h8, s8, dev_bf16(da), None, None, dh, dw)
    check_swiglu(h, da, np.ones(R), np.arange(R), R, h8, s8, a, dh, dw)
    bqm.bqm_swiglu_ckpt_bwd(h8, s8, dev_bf16(da), None, None, dh2)
    assert torch.equal(dh, dh2)


def test_swiglu_weight_gradient_of_large_factors():
    """da, g and u far apart in size, with a = silu(g) u and da a in the middle of the range:
    dtopk_w is the sum of da a, not an overflow of da silu(g) (above 2^129 each here)."""
    import torch
    log("swiglu, dtopk_w of large factors")
    bqm = _bqm()
    R, I = 3, 64
    g, u, da = (np.zeros((R, I)) for _ in range(3))
    g[0], u[0], da[0] = 2.0 ** 20, 2.0 ** -120, 2.0 ** 110
    g[1], u[1], da[1] = 40.0, 2.0 ** -100, 2.0 ** 124
    g[2], u[2], da[2] = 24.0, 2.0 ** -90, 1.5 * 2.0 ** 127
    da[:, ::3] *= -1
    h = np.concatenate([g, u], 1)
    h8, s8, a, dh = swiglu_buffers(R, I)
    dw = torch.empty(R, device=gpu())
    bqm.bqm_swiglu_ckpt_fwd(dev_bf16(h), h8, s8, a=a)
    bqm.bqm_swiglu_ckpt_bwd(h8, s8, dev_bf16(da), None, dev(np.full(R, 2.0 ** -40, np.float32)), dh, dw)
    check_swiglu(h, da, np.full(R, 2.0 ** -40), np.arange(R), R, h8, s8, a, dh, dw)
    assert np.isfinite(host(dw)).all()


def test_swiglu_every_block_maximum():
    """All bf16 magnitudes as a block's maximum, in the gate half and in the up half."""
    log("checkpoint block maxima")
    bqm = _bqm()
    rng = np.random.default_rng(6)
    top = (np.arange(1 << 15, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)
    R, I = 1 << 14, 32
    h = np.zeros((R, 2 * I))
    fin = np.where(np.isfinite(top), top, 1.0).reshape(R, 2)
    h[:, :I] = fin[:, :1] * rng.uniform(-1, 1, (R, I))
    h[:, I:] = fin[:, 1:] * rng.uniform(-1, 1, (R, I))
    h = bf16(h)
    h[:, 3], h[:, I + 5] = top.reshape(R, 2).T
    h8, s8, a, dh = swiglu_buffers(R, I)
    bqm.bqm_swiglu_ckpt_fwd(dev_bf16(h), h8, s8, a=a)
    c, s = mx.e4m3_checkpoint(h)
    assert (host(s8) == s).all()
    assert (host(h8) == c)[np.repeat(s != 255, 32, -1)].all()


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------
ROUTERS = [  # T, E, k, renorm, padded, masked, odd (duplicate and dropped indices)
    (1, 1, 1, False, False, 0, False),
    (1, 8, 2, True, False, 0, False),
    (7, 13, 3, False, True, 2, True),
    (64, 16, 16, True, False, 0, False),
    (300, 37, 4, True, True, 5, True),
    (515, 64, 8, False, True, 0, True),
    (1000, 128, 6, True, False, 8, False),
    (33, 250, 16, True, True, 7, True),
    (4099, 256, 8, False, False, 16, False),
    (129, 512, 8, True, False, 0, True),
    (70, 1000, 10, False, True, 100, False),
    (41, 1023, 3, True, False, 0, True),
    (200, 1024, 16, False, True, 0, True),
]


def router_case(T, E, k, padded, masked, odd):
    rng = np.random.default_rng([T, E, k])
    l = (rng.standard_normal((T, E)) * 3 + rng.standard_normal(E)).astype(np.float32)
    if masked:
        l[:, rng.permutation(E)[:masked]] = -np.inf
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    if odd:
        idx[0] = idx[0, 0]
        idx[T // 2, 0] = -1
        idx[T - 1, k - 1] = E
    dw = rng.standard_normal((T, k)).astype(np.float32)
    valid = None
    if padded:
        valid = (rng.random(T) < 0.7).astype(np.uint8) * rng.integers(1, 256, T).astype(np.uint8)
        l[valid == 0] = np.nan
        dw[valid == 0] = np.inf
    return l, idx, dw, valid


def run_router(l, idx, dw, valid, dloss, renorm, ws=None):
    import torch
    bqm = _bqm()
    T, E = l.shape
    counts = torch.full((E + 1,), -5, dtype=torch.int32, device=gpu())
    loss = torch.full((2,), 9.0, device=gpu())
    out = torch.full((T, E), 9.0, device=gpu())
    if ws is None:
        ws = torch.randint(0, 256, (bqm.bqm_router_loss_workspace_size(T, E),), dtype=torch.uint8, device=gpu())
    v = None if valid is None else dev(valid)
    bqm.bqm_router_loss(dev(l), dev(idx), v, counts, loss, ws)
    bqm.bqm_router_grad(dev(l), dev(idx), v, counts, None if dw is None else dev(dw),
                        None if dloss is None else dev(dloss), renorm, out)
    return counts, loss, out


@pytest.mark.parametrize("T,E,k,renorm,padded,masked,odd", ROUTERS)
def test_router_against_oracle(T, E, k, renorm, padded, masked, odd):
    import torch
    log(f"router T={T} E={E} k={k} renorm={renorm} padded={padded} masked={masked}")
    l, idx, dw, valid = router_case(T, E, k, padded, masked, odd)
    dloss = np.array([0.5, 0.25], np.float32)
    counts, loss, out = run_router(l, idx, dw, valid, dloss, renorm)
    c, lo = mx.router_loss(l, idx, valid)
    assert (host(counts) == c).all()
    within(host(loss), lo, 2.0 ** -18 * np.abs(lo) + 1e-30, "loss")
    g, size = mx.router_grad(l, idx, valid, c, dw, dloss.astype(np.float64), renorm)
    within(host(out), g, 2.0 ** -18 * size + 1e-30, "dlogits")
    if padded:
        assert (host(out)[valid == 0] == 0).all()
    again = run_router(l, idx, dw, valid, dloss, renorm)
    assert all(torch.equal(a, b) for a, b in zip((counts, loss, out), again)), "two calls differ"
    # each gradient alone
    for d, dl in ((dw, None), (None, dloss)):
        _, _, out = run_router(l, idx, d, valid, dl, renorm)
        g, size = mx.router_grad(l, idx, valid, c, np.zeros_like(dw) if d is None else d,
                                 np.zeros(2) if dl is None else dl.astype(np.float64), renorm)
        within(host(out), g, 2.0 ** -18 * size + 1e-30, "dlogits of one")


@pytest.mark.parametrize("E,k", [(3, 2), (13, 3), (21, 4), (37, 4), (60, 8), (100, 16), (250, 8), (1000, 4)])
def test_router_gradient_ignores_what_dropped_pairs_hold(E, k):
    """Indices outside [0, E), those among them that fall on a lane's unused places, with
    NaN and infinite gradients: the result is that of no gradient there."""
    import torch
    log(f"router, dropped pairs E={E} k={k}")
    T = 70
    l, idx, dw, _ = router_case(T, E, k, False, 0, False)
    rng = np.random.default_rng(E)
    drop = rng.random((T, k)) < 0.4
    beyond = np.array([-1, -E, E, E + 1, E + 2, E + 3, 1 << 30, -(1 << 31)])
    idx[drop] = beyond[rng.integers(0, len(beyond), drop.sum())]
    clean = np.where(drop, np.float32(0), dw)
    dw[drop] = np.array([np.nan, np.inf, -np.inf], np.float32)[rng.integers(0, 3, drop.sum())]
    dloss = np.array([0.5, 0.25], np.float32)
    for renorm in (False, True):
        c, _, out = run_router(l, idx, dw, None, dloss, renorm)
        _, _, want = run_router(l, idx, clean, None, dloss, renorm)
        assert torch.equal(out, want)
        g, size = mx.router_grad(l, idx, None, host(c), clean, dloss.astype(np.float64), renorm)
        within(host(out), g, 2.0 ** -18 * size + 1e-30, "dlogits")


@pytest.mark.parametrize("E", [5, 16, 30, 60, 128, 200, 256, 512, 1000])
@pytest.mark.parametrize("row", ["nan", "nan_and_off", "some"])
def test_router_losses_show_nan_logits(E, row):
    """A token that counts with NaN among its logits, whatever the others are (nothing but NaN,
    NaN and switched-off experts, finite ones): both losses are NaN, as their sums are, and so
    are the gradients of its logits; those of the other tokens' are not."""
    log(f"router, NaN logits E={E} {row}")
    T, k = 9, 2
    l, idx, dw, _ = router_case(T, E, k, False, 0, False)
    if row == "nan":
        l[4] = np.nan
    elif row == "nan_and_off":
        l[4] = -np.inf
        l[4, E // 2] = np.nan
    else:
        l[4, E // 2] = np.nan
    c, loss, out = run_router(l, idx, dw, None, np.ones(2, np.float32), False)
    assert host(c)[E] == T and np.isnan(host(loss)).all(), host(loss)
    nan = np.isnan(host(out)).all(1)
    assert nan[4] and not np.isnan(host(out)[np.arange(T) != 4]).any()
    c, loss, out = run_router(l, idx, dw, (np.arange(T) != 4).astype(np.uint8), np.ones(2, np.float32), False)
    assert np.isfinite(host(loss)).all() and np.isfinite(host(out)).all()


def test_router_batches_of_nothing():
    log("router, no tokens that count")
    E, k = 12, 2
    c, loss, out = run_router(np.zeros((0, E), np.float32), np.zeros((0, k), np.int32), np.zeros((0, k), np.float32),
                              None, np.ones(2, np.float32), False)
    assert (host(c) == 0).all() and (host(loss) == 0).all() and out.numel() == 0
    l = np.full((3, E), np.nan, np.float32)
    idx = np.zeros((3, k), np.int32)
    c, loss, out = run_router(l, idx, np.ones((3, k), np.float32), np.zeros(3, np.uint8), np.ones(2, np.float32), True)
    assert (host(c) == 0).all() and (host(loss) == 0).all() and (host(out) == 0).all()
    l[:] = -np.inf                              # tokens that count, with every expert off
    for renorm in (False, True):
        c, loss, out = run_router(l, idx, np.ones((3, k), np.float32), None, np.ones(2, np.float32), renorm)
        assert host(c)[0] == 6 and host(c)[E] == 3 and (host(loss) == 0).all() and (host(out) == 0).all()


def test_router_gradient_against_differences_of_its_own_loss():
    """Central differences of bqm_router_loss.  With step h the loss moves by 2 h g; its FP32
    rounding (2^-24 relative, twice) and the third-order term (h^2 / 6 times a third
    derivative of at most 32 times the loss's scale) bound what the quotient is off."""
    log("router gradient against differences")
    T, E, k, h = 3, 8, 2, 0.02
    l, idx, _, _ = router_case(T, E, k, False, 0, False)
    for which in (0, 1):
        dloss = np.zeros(2, np.float32)
        dloss[which] = 1.0
        _, base, out = run_router(l, idx, None, None, dloss, False)
        scale = max(1.0, float(host(base)[which]))
        tol = 2 * 2.0 ** -24 * scale / h + 32 * scale * h * h / 6
        for t in range(T):
            for e in range(E):
                lo, hi = l.copy(), l.copy()
                lo[t, e] -= np.float32(h)
                hi[t, e] += np.float32(h)
                step = float(hi[t, e]) - float(lo[t, e])
                d = (host(run_router(hi, idx, None, None, None, False)[1]) -
                     host(run_router(lo, idx, None, None, None, False)[1]))[which] / step
                assert abs(d - host(out)[t, e]) <= tol, (which, t, e)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Layer:
    """One MXFP4 expert layer's training step through the public entry points."""

    def __init__(self, T, E, k, H, I, seed=0, renorm=True):
        import torch
        bqm = _bqm()
        rng = np.random.default_rng([T, E, k, H, I, seed])
        self.T, self.E, self.k, self.H, self.I, self.renorm = T, E, k, H, I, renorm
        R = self.R = T * k
        d = gpu()
        self.x, self.dout = bf16(rng.standard_normal((T, H))), bf16(rng.standard_normal((T, H)))
        self.wgu, self.wdn = bf16(rng.standard_normal((E, 2 * I, H)) * 0.05), bf16(rng.standard_normal((E, H, I)) * 0.05)
        self.l = (rng.standard_normal((T, E)) * 2).astype(np.float32)
        self.l[:, 0] = -np.inf
        self.d_x, self.d_dout, self.d_l = dev_bf16(self.x), dev_bf16(self.dout), dev(self.l)
        self.q_gu, self.q_dn = quantize(self.wgu), quantize(self.wdn)
        e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=d)  # noqa: E731
        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        self.idx, self.w = e(T, k, dtype=i32), e(T, k, dtype=f32)
        self.perm, self.inv, self.off = e(R, dtype=i32), e(R, dtype=i32), e(E + 1, dtype=i32)
        self.pws = e(max(16, bqm.bqm_permute_workspace_size(T, E, k)), dtype=u8)
        self.rws = e(bqm.bqm_router_loss_workspace_size(T, E), dtype=u8)
        self.counts, self.loss = e(E + 1, dtype=i32), e(2, dtype=f32)
        self.xq = bqm.alloc_qtensor(bqm.FMT_MXFP4, 1, T, H)
        self.aq = bqm.alloc_qtensor(bqm.FMT_MXFP4, 1, R, I)
        self.h, self.y, self.da, self.dh, self.dxr = e(R, 2 * I), e(R, H), e(R, I), e(R, 2 * I), e(R, H)
        self.h8, self.s8 = e(R, 2 * I, dtype=u8), e(R, 2 * I // 32, dtype=u8)
        self.dw, self.dl = e(T, k, dtype=f32), e(T, E, dtype=f32)
        self.dloss = torch.tensor((0.01, 0.001), device=d)

    def step(self):
        b = _bqm()
        b.bqm_route(self.d_l, self.T, self.E, self.k, self.renorm, self.idx, self.w)
        b.bqm_permute(self.idx, self.T, self.E, self.k, self.perm, self.inv, self.off, self.pws)
        b.bqm_router_loss(self.d_l, self.idx, None, self.counts, self.loss, self.rws)
        b.bqm_quantize_mxfp4(self.d_x, self.xq)
        b.bqm_mxfp4_gemm(self.xq, self.q_gu, self.off, self.perm, self.k, self.h)
        b.bqm_swiglu_ckpt_fwd(self.h, self.h8, self.s8, aq=self.aq, n_rows=self.off[self.E:])
        b.bqm_mxfp4_gemm(self.aq, self.q_dn, self.off, None, 1, self.y)
        b.bqm_mxfp4_dgrad(self.q_dn, self.d_dout, self.off, self.perm, self.k, self.da)
        b.bqm_swiglu_ckpt_bwd(self.h8, self.s8, self.da, self.perm, self.w, self.dh, self.dw, n_rows=self.off[self.E:])
        b.bqm_mxfp4_dgrad(self.q_gu, self.dh, self.off, None, 1, self.dxr)
        b.bqm_router_grad(self.d_l, self.idx, None, self.counts, self.dw, self.dloss, self.renorm, self.dl)

    def outputs(self):
        return {n: getattr(self, n).clone() for n in ("idx", "w", "counts", "loss", "h", "h8", "s8", "y", "da", "dh",
                                                      "dxr", "dw", "dl")}


def check_layer(L):
    """Every stage against the oracle's arithmetic on the stage's own (bit-exact) inputs."""
    deq = mx.dequantize_mxfp4
    o = {n: host(t) for n, t in L.outputs().items()}
    perm, off, R = host(L.perm), host(L.off), L.R
    wgu, wdn = deq(*mx.quantize_mxfp4(L.wgu)), deq(*mx.quantize_mxfp4(L.wdn))
    T8 = 2.0 ** -8

    def prod(x, w, rows, n, what, got):
        ref, mag = mx.product(x, w, off, rows, np.zeros((R, w.shape[1])))
        within(got, ref, T8 * np.abs(ref) + n * 2.0 ** -23 * mag, what)

    prod(deq(*mx.quantize_mxfp4(L.x)), wgu, perm // L.k, L.H, "h", o["h"])
    q = deq(host(L.aq.codes)[0], host(L.aq.scales)[0])
    a = mx.swiglu(o["h"])
    # a went through bf16 and MXFP4: an element is within half a step of E2M1 (1 at most,
    # and 2 of saturation) of its block's scale
    sc = np.repeat(np.exp2(host(L.aq.scales)[0].astype(np.float64) - 127), 32, -1)
    within(q, a, 2.0 * sc + 2 * T8 * np.abs(a), "a in MXFP4")
    prod(q, wdn, np.arange(R), L.I, "y", o["y"])
    prod(L.dout, np.ascontiguousarray(wdn.transpose(0, 2, 1)), perm // L.k, L.H, "da", o["da"])
    check_swiglu(o["h"], o["da"], o["w"].reshape(-1), perm, off[L.E], L.h8, L.s8, dev_bf16(a), L.dh, L.dw)
    prod(o["dh"], np.ascontiguousarray(wgu.transpose(0, 2, 1)), np.arange(R), 2 * L.I, "dx rows", o["dxr"])
    c, lo = mx.router_loss(L.l, o["idx"])
    assert (o["counts"] == c).all() and (np.diff(off) == c[:L.E]).all()
    within(o["loss"], lo, 2.0 ** -18 * np.abs(lo), "losses")
    g, size = mx.router_grad(L.l, o["idx"], None, c, o["dw"], host(L.dloss), L.renorm)
    within(o["dl"], g, 2.0 ** -18 * size + 1e-30, "dlogits")


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 64, 32), (17, 16, 4, 320, 96), (300, 6, 2, 256, 160)])
def test_layer_step(T, E, k, H, I):
    log(f"layer T={T} E={E} k={k} H={H} I={I}")
    L = Layer(T, E, k, H, I)
    L.step()
    check_layer(L)


def test_layer_step_captured_and_replayed():
    import torch
    log("layer step in a graph")
    L = Layer(40, 12, 3, 256, 96)
    other = Layer(9, 12, 3, 256, 96, seed=1)
    L.step()
    other.step()
    torch.cuda.synchronize()
    want, want2 = L.outputs(), other.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        L.step()
    for _ in range(4):
        for n in want:
            getattr(L, n).zero_()
        graph.replay()
        other.step()
        torch.cuda.synchronize()
        assert all(torch.equal(v, want[n]) for n, v in L.outputs().items())
        assert all(torch.equal(v, want2[n]) for n, v in other.outputs().items())


def test_two_streams_at_once():
    import torch
    log("two layers on two streams")
    a, b = Layer(60, 10, 2, 192, 64), Layer(45, 10, 2, 192, 64, seed=3)
    a.step()
    b.step()
    torch.cuda.synchronize()
    wa, wb = a.outputs(), b.outputs()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(sa):
            a.step()
        with torch.cuda.stream(sb):
            b.step()
    torch.cuda.synchronize()
    assert all(torch.equal(v, wa[n]) for n, v in a.outputs().items())
    assert all(torch.equal(v, wb[n]) for n, v in b.outputs().items())


def test_binding_checks_every_tensor():
    """Each argument of each call in turn with another type, layout or size (nothing is
    launched: the checks come first)."""
    import torch
    log("binding checks")
    bqm = _bqm()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=gpu())  # noqa: E731
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    w, x = bqm.alloc_qtensor(bqm.FMT_MXFP4, 4, 64, 32), bqm.alloc_qtensor(bqm.FMT_MXFP4, 1, 8, 32)
    calls = [
        (bqm.bqm_mxfp4_gemm, [x, w, z(5, dtype=i32), z(8, dtype=i32), 1, z(8, 64)], (2, 3, 5)),
        (bqm.bqm_mxfp4_dgrad, [w, z(8, 64), z(5, dtype=i32), z(8, dtype=i32), 1, z(8, 32)], (1, 2, 3, 5)),
        (bqm.bqm_swiglu_ckpt_fwd, [z(4, 128), z(4, 128, dtype=u8), z(4, 4, dtype=u8), z(4, 64), None, z(1, dtype=i32)],
         (0, 1, 2, 3, 5)),
        (bqm.bqm_swiglu_ckpt_bwd, [z(4, 128, dtype=u8), z(4, 4, dtype=u8), z(4, 64), z(4, dtype=i32), z(4, dtype=f32),
                                   z(4, 128), z(4, dtype=f32), z(1, dtype=i32)], (0, 1, 2, 3, 4, 5, 6, 7)),
        (bqm.bqm_router_loss, [z(4, 8, dtype=f32), z(4, 2, dtype=i32), z(4, dtype=u8), z(9, dtype=i32), z(2, dtype=f32),
                               z(1 << 16, dtype=u8)], (0, 1, 2, 3, 4)),
        (bqm.bqm_router_grad, [z(4, 8, dtype=f32), z(4, 2, dtype=i32), z(4, dtype=u8), z(9, dtype=i32),
                               z(4, 2, dtype=f32), z(2, dtype=f32), 0, z(4, 8, dtype=f32)], (0, 1, 2, 3, 4, 5, 7)),
    ]
    for f, args, tensors in calls:
        f(*args)
        for i in tensors:
            t = args[i]
            wide = torch.zeros(*t.shape, 2, dtype=t.dtype, device=t.device)[..., 0]
            for other in (t.to(torch.float64), wide if t.numel() > 1 else None, t.cpu(),
                          None if t is args[0] or t.numel() < 2 else t.reshape(-1)[1:].clone()):
                if other is None:
                    continue
                if other.dim() < 2 <= t.dim() and f in (bqm.bqm_mxfp4_gemm, bqm.bqm_mxfp4_dgrad, bqm.bqm_swiglu_ckpt_bwd):
                    other = t[1:].clone()
                with pytest.raises((bqm.BQMError, ValueError, IndexError)):
                    f(*args[:i], other, *args[i + 1:])
    torch.cuda.synchronize()


def test_binding_refuses_another_device_and_host_workspaces(monkeypatch):
    import torch
    from bit_quantized_moe_amd import _lib
    log("binding, device checks")
    bqm = _bqm()
    x = torch.zeros((1, 8, 32), dtype=torch.bfloat16, device=gpu())
    q = bqm.alloc_qtensor(bqm.FMT_MXFP4, 1, 8, 32)
    l, idx = torch.zeros((4, 8), device=gpu()), torch.zeros((4, 2), dtype=torch.int32, device=gpu())
    counts, loss = torch.zeros(9, dtype=torch.int32, device=gpu()), torch.zeros(2, device=gpu())
    with pytest.raises(_lib.BQMError, match="ws: not a GPU tensor"):
        bqm.bqm_router_loss(l, idx, None, counts, loss, torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(_lib.BQMError, match="ws: not contiguous"):
        bqm.bqm_router_loss(l, idx, None, counts, loss, torch.zeros(1 << 17, dtype=torch.uint8, device=gpu())[::2])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: x.get_device() + 1)
    with pytest.raises(_lib.BQMError, match="x: on device"):
        bqm.bqm_quantize_mxfp4(x, q)
