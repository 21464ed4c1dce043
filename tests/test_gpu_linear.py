"""GPU parity of the dense product with its epilogue and of its gradients, against
oracle/linear.py (float64; for the larger sizes the same formulas in float64 on the GPU).

Tolerances, per element (bf16 rounds to within 2^-8 of a value, FP32 to within 2^-24):
* a product of C terms: they are exact in FP32, and at most C additions are off by one unit in
  the last place (2^-23) of a partial sum no larger than S, the sum of the terms' magnitudes
  (the bias among them): E = C 2^-23 S.
* act and act' of a value known exactly: with v s(t) (t = v, or 2 sqrt(2/pi) (v + 0.044715 v^3),
  formed with 6 roundings), e^-t is off by (8 |t| + 4) 2^-24 of itself, its reciprocal and the
  products by 8 more: (4 |t| + 16) 2^-23 of the terms' magnitudes.  Derivatives lie within
  [-0.13, 1.13], so E passes through an activation with a factor of 1.13.
* what is rounded to bf16 adds 2^-8 of the value, that is 2^-8 |ref| and 2^-8 of the rest.
* the bias gradient: M additions, M 2^-24 of the sum of magnitudes.
* adding to what the output holds: 2^-23 of both.
"""
import numpy as np
import pytest

from oracle import linear as oracle
from tests.gpu_util import gpu, log

pytestmark = pytest.mark.gpu

F8, F23, F24 = 2.0 ** -8, 2.0 ** -23, 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu_tanh"]


def _bqm():
    import bit_quantized_moe_amd as bqm
    return bqm


def act_id(name):
    return getattr(_bqm(), "ACT_" + name.upper())


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(dtype) if dtype is not None else t).to(gpu())


def bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def dev_bf16(a):
    import torch
    return None if a is None else dev(np.asarray(a, dtype=np.float32), torch.bfloat16)


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]}, {tol[bad][0]} allowed")


def empty(*s, dtype=None):
    import torch
    return torch.full(s, 77.0, dtype=dtype or torch.bfloat16, device=gpu())


def workspace(M, N, K):
    import torch
    n = _bqm().bqm_linear_workspace_size(M, N, K)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=gpu()) if n else None    # NaN where it is read unwritten


def eval_err(v, name, grad=False):
    """How far act(v) or act'(v) may be off, v exact."""
    if name in ("none", "relu"):
        return np.zeros_like(v)
    t = v if name == "silu" else 2 * oracle.C * (v + 0.044715 * v ** 3)
    s = oracle.sigmoid(t)
    slope = 1.0 if name == "silu" else 2 * oracle.C * (1 + 3 * 0.044715 * v * v)
    terms = s + np.abs(v) * s * (1 - s) * slope if grad else np.abs(v) * s
    # the difference 1 - s is formed with an absolute error of 2^-23
    more = np.abs(v) * s * slope * F23 if grad else 0.0
    return (4 * np.abs(t) + 16) * F23 * terms + more + 1e-36


def rounded(ref, err):
    return F8 * np.abs(ref) + (1 + F8) * err


def check_fwd(M, N, K, name, bias, residual, keep, seed=0, scale=1.0):
    rng = np.random.default_rng([M, N, K, seed])
    x, w = bf16(rng.standard_normal((M, K))), bf16(rng.standard_normal((N, K)) * scale / np.sqrt(K))
    b = bf16(rng.standard_normal(N)) if bias else None
    r = bf16(rng.standard_normal((M, N))) if residual else None
    y, z = empty(M, N), empty(M, N) if keep else None
    _bqm().bqm_linear_fwd(dev_bf16(x), dev_bf16(w), y, bias=dev_bf16(b), act=act_id(name), residual=dev_bf16(r), z=z,
                          ws=workspace(M, N, K))
    ry, rz, mag = oracle.fwd(x, w, b, name, r)
    e = (K + 1) * F23 * mag
    if keep:
        within(host(z), rz, rounded(rz, e), "z")
    err = (e if name == "none" else 1.13 * e + eval_err(rz, name)) + F23 * (np.abs(oracle.act(rz, name)) + np.abs(ry))
    within(host(y), ry, rounded(ry, err), "y")


def check_dgrad(M, N, K, name, add, seed=0):
    rng = np.random.default_rng([M, N, K, seed, 1])
    dz, w = bf16(rng.standard_normal((M, N))), bf16(rng.standard_normal((N, K)) / np.sqrt(N))
    zx = bf16(rng.standard_normal((M, K)) * 3) if name != "none" else None
    a = bf16(rng.standard_normal((M, K))) if add else None
    dx = empty(M, K)
    _bqm().bqm_linear_dgrad(dev_bf16(dz), dev_bf16(w), dx, zx=dev_bf16(zx), act=act_id(name), add=dev_bf16(a),
                            ws=workspace(M, N, K))
    ref, d, mag = oracle.dgrad(dz, w, zx, name, a)
    err = N * F23 * mag
    if name != "none":
        err = 1.13 * err + np.abs(d) * eval_err(zx, name, True)
    err = err + F23 * (np.abs(ref) + np.abs(ref - (0 if a is None else a)))
    within(host(dx), ref, rounded(ref, err), "dx")


def check_wgrad(M, N, K, accumulate, with_bias, seed=0):
    import torch
    rng = np.random.default_rng([M, N, K, seed, 2])
    dz, x = bf16(rng.standard_normal((M, N))), bf16(rng.standard_normal((M, K)))
    dw0, db0 = rng.standard_normal((N, K)).astype(np.float32), rng.standard_normal(N).astype(np.float32)
    dw, db = dev(dw0), dev(db0) if with_bias else None
    _bqm().bqm_linear_wgrad(dev_bf16(dz), dev_bf16(x), dw, dbias=db, accumulate=accumulate, ws=workspace(M, N, K))
    rw, mw, rb, mb = oracle.wgrad(dz, x)
    old_w, old_b = (dw0.astype(np.float64), db0.astype(np.float64)) if accumulate else (0 * rw, 0 * rb)
    within(host(dw), rw + old_w, M * F23 * mw + F23 * (np.abs(old_w) + np.abs(rw)) * accumulate, "dw")
    if with_bias:
        within(host(db), rb + old_b, M * F24 * mb + F23 * (np.abs(old_b) + np.abs(rb)) * accumulate, "db")
    assert dw.dtype == torch.float32


# one row and column of tiles and more, contractions of less than a step, one, parts of one
SHAPES = [(1, 8, 8), (1, 64, 64), (3, 16, 72), (2, 200, 56), (31, 72, 128), (32, 136, 120), (33, 264, 64), (63, 8, 520),
          (64, 128, 136), (65, 64, 192), (100, 56, 40), (127, 520, 200), (129, 264, 264), (200, 1040, 72), (257, 72, 1040),
          (300, 392, 648), (5, 2056, 1032), (16, 1032, 2056), (48, 528, 3080), (513, 8, 16),
          # few rows: contractions of several turns of the waves, columns past the last 16
          (1, 520, 4104), (2, 24, 1160), (4, 72, 2184), (3, 40, 3208), (4, 8, 8200), (8, 24, 4096), (7, 2056, 4104), (6, 40, 72),
          (8, 2048, 4104)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(M, N, K):
    log(f"forward {M} {N} {K}")
    for i, name in enumerate(ACTS):
        check_fwd(M, N, K, name, bias=i % 2 == 0, residual=i < 2, keep=i != 1, seed=i)
    check_fwd(M, N, K, "gelu_tanh", True, True, False, seed=9, scale=4.0)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_input_gradient(M, N, K):
    log(f"input gradient {M} {N} {K}")
    for i, name in enumerate(ACTS):
        check_dgrad(M, N, K, name, add=i % 2 == 1, seed=i)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_weight_gradient(M, N, K):
    log(f"weight gradient {M} {N} {K}")
    check_wgrad(M, N, K, False, True)
    check_wgrad(M, N, K, True, True)
    check_wgrad(M, N, K, True, False)


# sizes at which each tile occurs in each direction, with its last tile filled to each quarter,
# with the contraction in one part and in several, with and without whole rounds of tiles
LARGE = [(1111, 2848, 2080), (700, 4104, 520), (2050, 1048, 264), (4100, 512, 136), (150, 4096, 2048), (1000, 1000, 4104),
         (3000, 2056, 1032), (72, 6144, 2048), (8200, 2304, 96), (2817, 392, 2968), (8638, 6568, 72), (899, 1360, 4272),
         (436, 8896, 8304), (4159, 1336, 904), (1353, 4240, 960), (864, 1560, 5408), (258, 5752, 6120), (8778, 1720, 2928),
         (5051, 856, 1720), (4128, 7800, 1008), (3906, 1064, 8352), (1158, 2360, 6576), (1160, 2144, 7312), (1100, 40008, 72), (2100, 136, 40008),
         (5000, 70000, 64), (6515, 136, 6512), (8792, 3216, 136), (5927, 5312, 136)]


@pytest.mark.parametrize("M,N,K", LARGE)
def test_large(M, N, K):
    import torch
    log(f"large {M} {N} {K}")
    b = _bqm()
    g = torch.Generator(device=gpu()).manual_seed(M)
    rnd = lambda *s: torch.randn(s, generator=g, device=gpu()).to(torch.bfloat16)  # noqa: E731
    x, w, bias, res, dz = rnd(M, K), (rnd(N, K).float() / K ** 0.5).to(torch.bfloat16), rnd(N), rnd(M, N), rnd(M, N)
    ws = workspace(M, N, K)
    X, W, D = x.double(), w.double(), dz.double()

    def near(got, ref, err, what):
        bad = ~((got.double() - ref).abs() <= err)
        assert not bad.any(), f"{what}: {int(bad.sum())} outside, first at {bad.nonzero()[0].tolist()}"

    y, z = empty(M, N), empty(M, N)
    b.bqm_linear_fwd(x, w, y, bias=bias, act=b.ACT_RELU, residual=res, z=z, ws=ws)
    rz = X @ W.T + bias.double()
    e = (K + 1) * F23 * (X.abs() @ W.abs().T + bias.double().abs())
    near(z, rz, F8 * rz.abs() + 1.01 * e, "z")
    ry = rz.clamp(min=0) + res.double()
    near(y, ry, F8 * ry.abs() + 1.01 * (e + F23 * (rz.abs() + ry.abs())), "y")
    dx = empty(M, K)
    b.bqm_linear_dgrad(dz, w, dx, zx=x, act=b.ACT_RELU, add=x, ws=ws)
    d = D @ W
    rx = d * (X > 0) + X
    near(dx, rx, F8 * rx.abs() + 1.01 * (N * F23 * (D.abs() @ W.abs()) + F23 * (rx.abs() + d.abs())), "dx")
    dw, db = empty(N, K, dtype=torch.float32), empty(N, dtype=torch.float32)
    b.bqm_linear_wgrad(dz, x, dw, dbias=db, ws=ws)
    near(dw, D.T @ X, M * F23 * (D.T.abs() @ X.abs()), "dw")
    near(db, D.sum(0), M * F24 * D.abs().sum(0), "db")
    b.bqm_linear_wgrad(dz, x, dw, dbias=db, accumulate=True, ws=ws)
    near(dw, 2 * (D.T @ X), 2.01 * M * F23 * (D.T.abs() @ X.abs()), "dw, added")
    near(db, 2 * D.sum(0), 2.01 * M * F24 * D.abs().sum(0), "db, added")
    # the same bits again, without what changes nothing
    again, dx2, dw2 = empty(M, N), empty(M, K), empty(N, K, dtype=torch.float32)
    zero = torch.zeros_like(res), torch.zeros_like(bias), torch.zeros_like(x)
    b.bqm_linear_fwd(x, w, y, bias=zero[1], act=b.ACT_SILU, residual=zero[0], ws=ws)
    b.bqm_linear_fwd(x, w, again, act=b.ACT_SILU, z=z, ws=ws)
    assert torch.equal(again, y)
    for name in ("none", "silu", "gelu_tanh"):
        act = act_id(name)
        b.bqm_linear_fwd(x, w, y, bias=bias, act=act, ws=ws)
        s, slope = {"none": (1.0, 0.0), "silu": (torch.sigmoid(rz), 1.0),
                    "gelu_tanh": (torch.sigmoid(2 * oracle.C * (rz + 0.044715 * rz ** 3)), 0.0)}[name]
        # |2 sqrt(2/pi) (v + 0.044715 v^3)| is at most 1.6 |v| + 0.072 |v|^3
        t = 0.0 if name == "none" else rz.abs() if slope else 1.6 * rz.abs() + 0.072 * rz.abs() ** 3
        ry = rz * s
        near(y, ry, F8 * ry.abs() + 1.01 * (1.13 * e + (4 * t + 17) * F23 * ry.abs() + 1e-36), name)
        b.bqm_linear_dgrad(dz, w, dx, zx=x, act=act, add=zero[2], ws=ws)
        b.bqm_linear_dgrad(dz, w, dx2, zx=x, act=act, ws=ws)
        assert torch.equal(dx, dx2)
        v = X if name != "none" else 0 * X
        s = torch.sigmoid(v if slope else 2 * oracle.C * (v + 0.044715 * v ** 3))
        q = v.abs() * s * (1 - s) * (1.0 if slope else 2 * oracle.C * (1 + 3 * 0.044715 * v * v))
        g = 1.0 if name == "none" else s + v.sign() * q
        t = v.abs() if slope else 1.6 * v.abs() + 0.072 * v.abs() ** 3
        off = 0.0 if name == "none" else (4 * t + 16) * F23 * (s + q) + q / (1 - s) * F23 + 1e-36
        near(dx, d * g, F8 * (d * g).abs() + 1.01 * (1.13 * N * F23 * (D.abs() @ W.abs()) + d.abs() * off + F23 * (d * g).abs()), name)
    b.bqm_linear_dgrad(dz, w, dx, add=x, ws=ws)
    near(dx, d + X, F8 * (d + X).abs() + 1.01 * (N * F23 * (D.abs() @ W.abs()) + F23 * (d + X).abs()), "dx, added to")
    b.bqm_linear_wgrad(dz, x, dw, ws=ws)
    b.bqm_linear_wgrad(dz, x, dw2, ws=ws)
    assert torch.equal(dw2, dw)


def test_past_four_gigabytes():
    """Inputs and outputs of 400000 x 6144: byte and element offsets pass 32 bits."""
    import torch
    log("past 4 GiB")
    b = _bqm()
    M, N, K = 400003, 64, 6144
    g = torch.Generator(device=gpu()).manual_seed(1)
    x = torch.randn((M, K), generator=g, device=gpu(), dtype=torch.bfloat16)
    w = (torch.randn((N, K), generator=g, device=gpu()) / 64).to(torch.bfloat16)
    ws = workspace(M, N, K)
    some = torch.cat([torch.arange(0, M, 4999, device=gpu()), torch.tensor([M - 1], device=gpu())])
    y = b.bqm_linear_fwd(x, w, empty(M, N), ws=ws)
    X, W = x[some].double(), w.double()
    ref = X @ W.T
    assert ((y[some].double() - ref).abs() <= F8 * ref.abs() + 1.01 * K * F23 * (X.abs() @ W.abs().T)).all()
    dx = b.bqm_linear_dgrad(y, w, empty(M, K), zx=x, act=b.ACT_RELU, ws=ws)
    D = y[some].double()
    ref = (D @ W) * (X > 0)
    assert ((dx[some].double() - ref).abs() <= F8 * ref.abs() + 1.01 * N * F23 * (D.abs() @ W.abs())).all()
    dw = b.bqm_linear_wgrad(y, x, empty(N, K, dtype=torch.float32), ws=ws)
    ref, mag = torch.zeros((N, K), dtype=torch.float64, device=gpu()), torch.zeros((N, K), dtype=torch.float64, device=gpu())
    for i in range(0, M, 50000):
        D, X = y[i:i + 50000].double(), x[i:i + 50000].double()
        ref += D.T @ X
        mag += D.T.abs() @ X.abs()
    assert ((dw.double() - ref).abs() <= M * F23 * mag).all()


def test_most_rows():
    """2^30 - 1 rows, nearly all zeros: whole numbers, exact in any order."""
    import torch
    log("most rows")
    b = _bqm()
    M, N, K = (1 << 30) - 1, 8, 8
    g = torch.Generator(device=gpu()).manual_seed(2)
    at = torch.cat([torch.randint(0, M, (4000,), generator=g, device=gpu()), torch.tensor([0, M - 70, M - 64, M - 1], device=gpu())]).unique()
    some = lambda: torch.randint(-3, 4, (len(at), 8), generator=g, device=gpu()).bfloat16()  # noqa: E731
    x, dz = (torch.zeros((M, 8), dtype=torch.bfloat16, device=gpu()) for _ in range(2))
    x[at], dz[at] = some(), some()
    w = some()[:8].contiguous()
    ws = workspace(M, N, K)
    X, D = x[at].double(), dz[at].double()
    dw, db = empty(N, K, dtype=torch.float32), empty(N, dtype=torch.float32)
    b.bqm_linear_wgrad(dz, x, dw, dbias=db, ws=ws)
    assert torch.equal(dw.double(), D.T @ X) and torch.equal(db.double(), D.sum(0))
    for product, a, ref in ((b.bqm_linear_fwd, x, X @ w.double().T), (b.bqm_linear_dgrad, dz, D @ w.double())):
        out = product(a, w, torch.full_like(x, 5.0), ws=ws)
        assert torch.equal(out[at].double(), ref)
        out[at] = 0
        assert not out.any()
        del out


def test_infinities_of_the_last_step():
    """Where the last step overlaps the one before, an infinity is counted once (0 times it
    would be NaN)."""
    import torch
    log("infinities")
    b = _bqm()
    for K in (72, 136, 200):
        x, w = torch.ones((2, K), device=gpu()).bfloat16(), torch.ones((16, K), device=gpu()).bfloat16()
        x[1, K - 60] = float("inf")
        w[3, K - 61] = -float("inf")
        y = host(b.bqm_linear_fwd(x, w, empty(2, 16), ws=workspace(2, 16, K)))
        assert (np.delete(y[0], 3) == K).all() and y[0, 3] == -np.inf and (np.delete(y[1], 3) == np.inf).all()
        assert np.isnan(y[1, 3])
    for M in (65, 100, 127):
        dz, x = torch.ones((M, 16), device=gpu()).bfloat16(), torch.ones((M, 8), device=gpu()).bfloat16()
        dz[M - 60, 5] = float("inf")
        dw = host(b.bqm_linear_wgrad(dz, x, empty(16, 8, dtype=torch.float32), ws=workspace(M, 16, 8)))
        assert (dw[5] == np.inf).all() and (np.delete(dw, 5, 0) == M).all()


@pytest.mark.parametrize("M,N,K", [(40, 256, 512), (3, 64, 64), (300, 1024, 2048)])
def test_in_place(M, N, K):
    """The residual's tensor as y, and add's as dx."""
    import torch
    log(f"in place {M} {N} {K}")
    b = _bqm()
    rng = np.random.default_rng(M)
    x, w, r, dz, a = (dev_bf16(rng.standard_normal(s)) for s in ((M, K), (N, K), (M, N), (M, N), (M, K)))
    ws = workspace(M, N, K)
    y = b.bqm_linear_fwd(x, w, empty(M, N), act=b.ACT_SILU, residual=r, ws=ws)
    assert torch.equal(b.bqm_linear_fwd(x, w, r, act=b.ACT_SILU, residual=r, ws=ws), y)
    dx = b.bqm_linear_dgrad(dz, w, empty(M, K), add=a, ws=ws)
    assert torch.equal(b.bqm_linear_dgrad(dz, w, a, add=a, ws=ws), dx)


def test_no_rows():
    import torch
    log("no rows")
    b = _bqm()
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=gpu())  # noqa: E731
    w = e(16, 24)
    assert b.bqm_linear_workspace_size(0, 16, 24) == 0
    b.bqm_linear_fwd(e(0, 24), w, e(0, 16))
    b.bqm_linear_dgrad(e(0, 16), w, e(0, 24))
    dw, db = empty(16, 24, dtype=torch.float32), empty(16, dtype=torch.float32)
    b.bqm_linear_wgrad(e(0, 16), e(0, 24), dw, dbias=db, accumulate=True)
    assert (dw == 77).all() and (db == 77).all()
    b.bqm_linear_wgrad(e(0, 16), e(0, 24), dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("name", ACTS[1:])
@pytest.mark.parametrize("n", [1, 7, 8, 2047, 2048, 2049, 100003])
def test_act_grad(name, n):
    log(f"act_grad {name} {n}")
    b = _bqm()
    rng = np.random.default_rng(n)
    dy, z = bf16(rng.standard_normal(n)), bf16(rng.standard_normal(n) * 4)
    # far from zero, where the sigmoid is 0 or 1, and where squares and cubes leave FP32
    far = np.array([0.0, -0.0, 15.5, -15.5, 16.5, -16.5, 40.0, -40.0, 87.0, -88.0, -89.0, 200.0, -200.0, 1e13, -1e13, 3e38, -3e38])
    z[: min(n, len(far))] = bf16(far)[:n]
    d_dy, d_z = dev_bf16(dy), dev_bf16(z)
    dz = b.bqm_act_grad(d_dy, d_z, act_id(name), empty(n))
    # beyond |z| = 80 the derivative is within 81 e^-80 < 2^-100 of 0 or 1, here as at 80
    near = np.clip(z, -80.0, 80.0)
    ref = dy * oracle.act_grad(near, name)
    err = np.abs(dy) * (eval_err(near, name, True) + 2.0 ** -99 * (np.abs(z) > 80)) + F23 * np.abs(ref)
    within(host(dz), ref, rounded(ref, err), "dz")
    import torch
    for alias in (d_dy, d_z):
        a, c = (alias.clone(), d_z) if alias is d_dy else (d_dy, alias.clone())
        assert torch.equal(b.bqm_act_grad(a, c, act_id(name), a if alias is d_dy else c), dz)


def test_activations_far_from_zero():
    """The forward's activations on the same values (a product with one 1 in each row)."""
    import torch
    log("activations far from zero")
    b = _bqm()
    v = np.zeros(24)
    v[:17] = bf16(np.array([0.0, -0.0, 15.5, -15.5, 16.5, -16.5, 40.0, -40.0, 87.0, -88.0, -89.0, 200.0, -200.0, 1e13, -1e13, 3e38, -3e38]))
    x, w = dev_bf16(np.ones((1, 8)) * (np.arange(8) == 0)), np.zeros((24, 8))
    w[:, 0] = v
    for name in ACTS[1:]:
        y = host(b.bqm_linear_fwd(x, dev_bf16(w), empty(1, 24), act=act_id(name)))[0]
        # below -80 the activation is within 80 e^-80 < 2^-100 of 0, here as at -80
        near = np.clip(v, -80.0, 80.0)
        ref = np.where(v > 80, v, oracle.act(near, name))
        within(y, ref, rounded(ref, eval_err(near, name) + 2.0 ** -99 * (v < -80)) + F8 * np.abs(ref), name)
    assert torch.isfinite(x).all()


@pytest.mark.parametrize("name", ACTS[1:])
def test_nan_and_infinity_through_activations(name):
    """A NaN pre-activation shows in the output and in the gradient; infinities have the limits'
    values where FP32 forms them; ReLU's gradient passes nothing where it is off."""
    import torch
    log(f"NaN and infinity {name}")
    b = _bqm()
    a, nan, inf = act_id(name), float("nan"), float("inf")
    for M in (2, 40):       # by the forward of few rows, and by tiles
        x = torch.zeros((M, 64), device=gpu()).bfloat16()
        w, bias = torch.ones((16, 64), device=gpu()).bfloat16(), torch.zeros(16, device=gpu()).bfloat16()
        bias[3], bias[4], bias[5] = nan, inf, -3.0
        y = b.bqm_linear_fwd(x, w, empty(M, 16), bias=bias, act=a, ws=workspace(M, 16, 64))
        assert y[:, 3].isnan().all() and (y[:, 4] == inf).all() and not y[:, 5].isnan().any() and (y[:, 6:] == 0).all()
        z = torch.zeros((M, 64), device=gpu()).bfloat16()
        z[:, 3], z[:, 4], z[:, 5], z[:, 6] = nan, 100.0, -100.0, -100.0
        dz = torch.zeros((M, 16), device=gpu()).bfloat16()
        dz[:, 0] = 1
        v = torch.ones((16, 64), device=gpu()).bfloat16()
        v[0, 6] = inf
        dx = b.bqm_linear_dgrad(dz, v, empty(M, 64), zx=z, act=a, ws=workspace(M, 16, 64))
        dy = torch.ones((M, 64), device=gpu()).bfloat16()
        dy[:, 6] = inf
        for got in (dx, b.bqm_act_grad(dy, z, a, empty(M, 64)), b.bqm_act_grad(dy[:, :7].contiguous(), z[:, :7].contiguous(), a, empty(M, 7))):
            assert (got[:, 3] == 1).all() if name == "relu" else got[:, 3].isnan().all()
            assert (got[:, 4] == 1).all() and (got[:, 5].abs() < 1e-30).all()
            assert name != "relu" or (got[:, 6] == 0).all()


def test_gradients_are_the_differences():
    """<dy, (y(p + h d) - y(p - h d)) / 2 h> of the oracle's forward against the GPU's gradients of
    x, w and b in the direction d, through an activation before and one behind the layer."""
    import torch
    log("gradients against differences")
    b = _bqm()
    M, N, K = 9, 40, 72
    rng = np.random.default_rng(3)
    zx, w, bias, dy = (rng.standard_normal(s) for s in ((M, K), (N, K), (N,), (M, N)))
    zx, w, bias, dy = bf16(zx), bf16(w / 8), bf16(bias), bf16(dy)
    x = bf16(oracle.act(zx, "silu"))
    # the backward through the layer's own activation, as dz, then both products
    _, z, _ = oracle.fwd(x, w, bias, "gelu_tanh", None)
    zb = bf16(z)
    dz = b.bqm_act_grad(dev_bf16(dy), dev_bf16(zb), b.ACT_GELU_TANH, empty(M, N))
    dx = b.bqm_linear_dgrad(dz, dev_bf16(w), empty(M, K), zx=dev_bf16(zx), act=b.ACT_SILU, ws=workspace(M, N, K))
    dw, db = empty(N, K, dtype=torch.float32), empty(N, dtype=torch.float32)
    b.bqm_linear_wgrad(dz, dev_bf16(x), dw, dbias=db, ws=workspace(M, N, K))

    def loss(zx_, w_, b_, xs=None):
        return (dy * oracle.fwd(oracle.act(zx_, "silu") if xs is None else xs, w_, b_, "gelu_tanh", None)[0]).sum()

    h = 1e-4
    for what, g, d, f in [
        ("zx", dx, rng.standard_normal((M, K)), lambda s, d: loss(zx + s * d, w, bias)),
        ("w", dw, rng.standard_normal((N, K)), lambda s, d: loss(zx, w + s * d, bias, x)),
        ("b", db, rng.standard_normal(N), lambda s, d: loss(zx, w, bias + s * d, x)),
    ]:
        num, ana = (f(h, d) - f(-h, d)) / (2 * h), (host(g) * d).sum()
        # z and x in bf16 (2^-8 of a value, through second derivatives below 2), dz and dx rounded
        # once each: every factor of every term is off by at most 4 * 2^-8 of its size
        W, X = np.abs(w), np.abs(x)
        size = {"zx": lambda: (np.abs(dy) @ W * np.abs(d)).sum() * 1.13 ** 2,
                "w": lambda: (np.abs(dy).T @ X * np.abs(d)).sum() * 1.13,
                "b": lambda: (np.abs(dy).sum(0) * np.abs(d)).sum() * 1.13}[what]()
        mag = 1 + np.abs(z).max()
        assert abs(num - ana) <= 8 * F8 * mag * size, (what, num, ana)


def test_binding_checks_every_tensor():
    import torch
    log("binding checks")
    b = _bqm()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=gpu())  # noqa: E731
    f32, u8 = torch.float32, torch.uint8
    ws = z(1 << 16, dtype=u8)
    calls = [
        (lambda x, w, y, bias, r, zz, ws: b.bqm_linear_fwd(x, w, y, bias=bias, act=1, residual=r, z=zz, ws=ws),
         [z(4, 64), z(16, 64), z(4, 16), z(16), z(4, 16), z(4, 16), ws]),
        (lambda dz, w, dx, zx, a, ws: b.bqm_linear_dgrad(dz, w, dx, zx=zx, act=1, add=a, ws=ws),
         [z(4, 16), z(16, 64), z(4, 64), z(4, 64), z(4, 64), ws]),
        (lambda dz, x, dw, db, ws: b.bqm_linear_wgrad(dz, x, dw, dbias=db, ws=ws),
         [z(4, 16), z(4, 64), z(16, 64, dtype=f32), z(16, dtype=f32), ws]),
        (lambda dy, zz, dz: b.bqm_act_grad(dy, zz, 1, dz), [z(4, 16), z(4, 16), z(4, 16)]),
    ]
    for f, args in calls:
        f(*args)
        for i, t in enumerate(args):
            wide = torch.zeros(*t.shape, 2, dtype=t.dtype, device=t.device)[..., 0]
            short = None if t.dtype is u8 else t[1:].clone()
            for other in (t.to(torch.float64), wide, t.cpu(), short):
                if other is None:
                    continue
                with pytest.raises((b.BQMError, ValueError)):
                    f(*args[:i], other, *args[i + 1:])
    torch.cuda.synchronize()


@pytest.mark.parametrize("most,N,K", [(1024, 4096, 6144), (600, 2056, 3080), (16384, 264, 264)])
def test_one_workspace_for_every_batch(most, N, K):
    """A workspace made for the largest batch serves the smaller ones, with the same bits as any other."""
    import torch
    log(f"one workspace {most} {N} {K}")
    b = _bqm()
    g = torch.Generator(device=gpu()).manual_seed(most)
    rnd = lambda *s: torch.randn(s, generator=g, device=gpu()).to(torch.bfloat16)  # noqa: E731
    x, w, dz, ws = rnd(most, K), rnd(N, K), rnd(most, N), workspace(most, N, K)
    larger = torch.full((ws.numel() + 4096,), 0xFF, dtype=torch.uint8, device=gpu())
    X, W, D = x.double(), w.double(), dz.double()

    def near(got, ref, err):
        assert ((got.double() - ref).abs() <= err).all()

    for M in [m for m in (1, 8, 9, 37, 100, 300, 500, 512, 513, 600, 1000, 1024, 8192, 16384) if m <= most]:
        xs, ds = x[:M], dz[:M]
        out = [[b.bqm_linear_fwd(xs, w, empty(M, N), ws=s), b.bqm_linear_dgrad(ds, w, empty(M, K), ws=s),
                b.bqm_linear_wgrad(ds, xs, empty(N, K, dtype=torch.float32), ws=s)] for s in (ws, larger)]
        assert all(torch.equal(p, q) for p, q in zip(*out)), M
        y, dx, dw = out[0]
        ref = X[:M] @ W.T
        near(y, ref, F8 * ref.abs() + 1.01 * K * F23 * (X[:M].abs() @ W.abs().T))
        ref = D[:M] @ W
        near(dx, ref, F8 * ref.abs() + 1.01 * N * F23 * (D[:M].abs() @ W.abs()))
        near(dw, D[:M].T @ X[:M], M * F23 * (D[:M].abs().T @ X[:M].abs()))


@pytest.mark.parametrize("name", ACTS[1:])
def test_gradients_along_themselves(name):
    """Differences of the oracle's forward along the signs of each gradient, where all terms add up,
    so that what is allowed (each element's rounding, as in the tests above) is small beside them.
    The two steps apart, each on the bf16 values it is given: z to act(z), and (zx, w, b) to
    act(zx) w^T + b.  Third derivatives of the activations stay below 4: central differences with
    h = 1e-4 are off by less than 1e-8 of the sum of the weights; float64 sums by less than 1e-7."""
    import torch
    log(f"gradients along themselves {name}")
    b = _bqm()
    M, N, K, h = 9, 40, 72, 1e-4
    rng = np.random.default_rng(17)
    z, zx, dy, dz, x = (bf16(rng.standard_normal(s)) for s in ((M, N), (M, K), (M, N), (M, N), (M, K)))
    w, bias = bf16(rng.standard_normal((N, K)) / 8), bf16(rng.standard_normal(N))
    assert min(np.abs(z).min(), np.abs(zx).min()) > 2 * h      # off ReLU's corner
    a = act_id(name)
    g_z = b.bqm_act_grad(dev_bf16(dy), dev_bf16(z), a, empty(M, N))
    g_zx = b.bqm_linear_dgrad(dev_bf16(dz), dev_bf16(w), empty(M, K), zx=dev_bf16(zx), act=a, ws=workspace(M, N, K))
    g_w, g_b = empty(N, K, dtype=torch.float32), empty(N, dtype=torch.float32)
    b.bqm_linear_wgrad(dev_bf16(dz), dev_bf16(x), g_w, dbias=g_b, ws=workspace(M, N, K))
    D, W = np.abs(dz), np.abs(w)
    ref_z = dy * oracle.act_grad(z, name)
    ref_zx, d, mag = oracle.dgrad(dz, w, zx, name, None)
    rw, mw, rb, mb = oracle.wgrad(dz, x)
    layer = lambda zx_, w_, b_: (dz * (oracle.act(zx_, name) @ w_.T + b_)).sum()  # noqa: E731
    plain = lambda w_, b_: (dz * (x @ w_.T + b_)).sum()  # noqa: E731
    for what, got, ref, f, err, weights in [
        ("z", g_z, ref_z, lambda s: (dy * oracle.act(z + s, name)).sum(),
         rounded(ref_z, np.abs(dy) * eval_err(z, name, True) + F23 * np.abs(ref_z)), np.abs(dy)),
        ("zx", g_zx, ref_zx, lambda s: layer(zx + s, w, bias),
         rounded(ref_zx, 1.13 * N * F23 * mag + np.abs(d) * eval_err(zx, name, True) + 2 * F23 * np.abs(ref_zx)), D @ W),
        ("w", g_w, rw, lambda s: plain(w + s, bias), M * F23 * mw, mw),
        ("b", g_b, rb, lambda s: plain(w, bias + s), M * F24 * mb, mb),
    ]:
        step = np.sign(ref)
        num, ana = (f(h * step) - f(-h * step)) / (2 * h), (host(got) * step).sum()
        allowed = err.sum() + 2e-7 * weights.sum()
        assert allowed < 0.01 * np.abs(ref).sum() and abs(num - np.abs(ref).sum()) < 2e-7 * weights.sum(), what
        assert abs(num - ana) <= allowed, (what, num, ana, allowed)


def test_past_four_gigabytes_exactly():
    """Whole numbers of up to 3 in 400003 x 6144: every product and sum is exact (below 2^24), so
    each row of the result and each row's part of the gradients counts."""
    import torch
    log("past 4 GiB, whole numbers")
    b = _bqm()
    M, N, K = 400003, 64, 6144
    g = torch.Generator(device=gpu()).manual_seed(4)
    some = lambda *s: torch.randint(-3, 4, s, generator=g, device=gpu(), dtype=torch.int8).bfloat16()  # noqa: E731
    x, w, dz = some(M, K), some(N, K), some(M, N)
    ws = workspace(M, N, K)
    y = b.bqm_linear_fwd(x, w, empty(M, N), ws=ws)
    dx = b.bqm_linear_dgrad(dz, w, empty(M, K), ws=ws)
    dw, db = empty(N, K, dtype=torch.float32), empty(N, dtype=torch.float32)
    b.bqm_linear_wgrad(dz, x, dw, dbias=db, ws=ws)
    W, ref = w.double(), torch.zeros((N, K), dtype=torch.float64, device=gpu())
    for i in range(0, M, 50000):
        X, D = x[i:i + 50000].double(), dz[i:i + 50000].double()
        assert torch.equal(y[i:i + 50000], (X @ W.T).bfloat16()), i
        assert torch.equal(dx[i:i + 50000], (D @ W).bfloat16()), i
        ref += D.T @ X
    assert torch.equal(dw.double(), ref)
    assert torch.equal(db.double(), dz.double().sum(0))


# sizes at which workgroups walk more than one tile, or a tile and a part of one: each tile in each
# direction where the plan does so, with last steps that are whole and that are not (LARGE has some
# of these only; test_linear_plan.py holds them to the plan)
ROUNDS = [(7286, 3224, 1344), (1556, 4984, 2416), (5874, 608, 2848), (2325, 2160, 3320), (4078, 1704, 240),
          (9239, 896, 800), (1318, 1120, 5568), (1173, 3008, 3248), (10956, 2584, 288), (9, 59000, 896), (10, 39776, 864),
          (10, 33608, 1920), (9, 37664, 2144), (1088, 3104, 2496), (642, 1152, 6752), (7872, 32824, 8), (7218, 33072, 8),
          (11244, 64, 1320), (9258, 72, 1608), (1264, 2880, 6752), (10980, 2584, 656), (11373, 1304, 64), (10963, 1288, 72),
          (4615, 3408, 896), (10053, 1544, 800), (64, 3216, 4944), (70, 37928, 264), (3328, 33512, 240), (2071, 64, 7376),
          (6530, 448, 2456), (331, 33616, 896), (64, 33176, 432), (640, 2232, 7280), (9, 36832, 64), (9, 32856, 72),
          (11, 33712, 768), (11, 34504, 656), (4544, 37408, 8), (1775, 32984, 8), (10979, 8, 264), (9, 32776, 8), (2049, 2056, 32)]


@pytest.mark.parametrize("M,N,K", ROUNDS)
def test_large_in_rounds(M, N, K):
    test_large(M, N, K)
