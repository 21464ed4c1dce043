"""GPU parity of the rows between token order and expert order, against oracle/rows.py.

Tolerances, per element (bf16 rounds to within 2^-8 of a value, FP32 to within 2^-24):
* copied rows: equal.
* combine: k products and k + 1 additions, each within 2^-24 of a value no larger than S = the
  sum of the terms' magnitudes: 2^-8 |ref| + (2 k + 1) 2^-24 S (2^-8 of the rounded sum, which
  is 2^-8 |ref| but for a part in 2^16: 2^-23 S more).
* dy: one product, then bf16: (2^-8 + 2^-23) |ref|.
* the weights' gradient: H exact products, H additions of partial sums no larger than S: H 2^-24 S.
"""
import numpy as np
import pytest

from oracle import rows as oracle
from tests.gpu_util import gpu, log

pytestmark = pytest.mark.gpu

F8, F24 = 2.0 ** -8, 2.0 ** -24


def _bqm():
    import bit_quantized_moe_amd as bqm
    return bqm


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(dtype) if dtype is not None else t).to(gpu())


def bf16(a):
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


def places(rng, T, k, kind):
    """inv [T, k] and the number of rows that hold data."""
    R = T * k
    inv = rng.permutation(R).astype(np.int32).reshape(T, k)
    if kind == "all":
        return inv, None
    if kind == "none":
        return inv, 0
    # places behind the live rows, and places that are no rows at all
    inv[rng.random((T, k)) < 0.1] = -1
    inv[rng.random((T, k)) < 0.05] = R
    inv[rng.random((T, k)) < 0.05] = 2 ** 31 - 1
    inv[rng.random((T, k)) < 0.05] = -2 ** 31
    return inv, int(R * 0.8)


SHAPES = [(1, 1, 1), (1, 8, 6144), (3, 2, 7), (5, 3, 8), (7, 16, 64), (33, 9, 72), (40, 17, 24), (257, 6, 256), (65, 4, 264),
          (130, 8, 2080), (9, 5, 4104), (4, 2, 8200), (6, 3, 601), (11, 1, 33), (300, 2, 16)]


class Case:
    def __init__(self, T, k, H, kind, seed=0):
        import torch
        rng = np.random.default_rng([T, k, H, seed])
        R = T * k
        self.T, self.k, self.H, self.R = T, k, H, R
        self.inv, live = places(rng, T, k, kind)
        self.n = R if live is None else live
        self.x, self.dout, self.res = (bf16(rng.standard_normal((T, H))) for _ in range(3))
        self.y = bf16(rng.standard_normal((R, H)))
        self.y[self.n:] = np.nan                    # what stands behind the live rows is not read
        self.w = rng.standard_normal((T, k)).astype(np.float32)
        self.d_inv = dev(self.inv)
        # as a view of a larger tensor, which starts at a multiple of 4 bytes only
        self.d_n = None if live is None else dev(np.array([7, live], dtype=np.int32))[1:]
        self.d_x, self.d_dout, self.d_res, self.d_y = dev_bf16(self.x), dev_bf16(self.dout), dev_bf16(self.res), dev_bf16(self.y)
        self.d_w = dev(self.w)
        self.empty = lambda *s, dtype=torch.bfloat16: torch.full(s, 77.0, dtype=dtype, device=gpu())


@pytest.mark.parametrize("kind", ["all", "dropped", "none"])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_against_oracle(T, k, H, kind):
    import torch
    log(f"rows T={T} k={k} H={H} {kind}")
    b = _bqm()
    c = Case(T, k, H, kind)
    mark = np.full((c.R, H), 77.0)
    rows = b.bqm_dispatch(c.d_x, c.d_inv, c.empty(c.R, H), n_rows=c.d_n)
    assert (host(rows) == oracle.dispatch(c.x, c.inv, c.n, mark)).all()
    for w, res in ((c.w, c.res), (None, None), (c.w, None), (None, c.res)):
        out = b.bqm_combine(c.d_y, c.d_inv, c.empty(T, H), topk_w=None if w is None else c.d_w,
                            residual=None if res is None else c.d_res, n_rows=c.d_n)
        ref, mag = oracle.combine(c.y, c.inv, c.n, w, res)
        within(host(out), ref, F8 * np.abs(ref) + (2 * k + 3) * F24 * mag, "out")
    for w in (c.w, None):
        dy, dw = c.empty(c.R, H), c.empty(T, k, dtype=torch.float32)
        d_w = None if w is None else c.d_w
        b.bqm_combine_grad(c.d_dout, c.d_inv, y=c.d_y, topk_w=d_w, dy=dy, dtopk_w=dw, n_rows=c.d_n)
        rdy, rdw, mag = oracle.combine_grad(c.dout, c.y, c.inv, c.n, w, mark)
        within(host(dy), rdy, np.where(rdy == 77.0, 0.0, (F8 + 2 * F24) * np.abs(rdy)), "dy")
        within(host(dw), rdw, H * F24 * mag, "dtopk_w")
        # one of the two alone gives the same bits
        one, two = c.empty(c.R, H), c.empty(T, k, dtype=torch.float32)
        b.bqm_combine_grad(c.d_dout, c.d_inv, topk_w=d_w, dy=one, n_rows=c.d_n)
        b.bqm_combine_grad(c.d_dout, c.d_inv, y=c.d_y, topk_w=d_w, dtopk_w=two, n_rows=c.d_n)
        assert torch.equal(one, dy) and torch.equal(two, dw)


@pytest.mark.parametrize("T,k,H", [(50, 3, 328), (21, 2, 40), (13, 4, 5)])
def test_in_place(T, k, H):
    """The residual's tensor as the output, and y's as dy."""
    import torch
    log(f"in place {T} {k} {H}")
    b = _bqm()
    c = Case(T, k, H, "dropped")
    out = b.bqm_combine(c.d_y, c.d_inv, c.empty(T, H), topk_w=c.d_w, residual=c.d_res, n_rows=c.d_n)
    again = c.d_res.clone()
    b.bqm_combine(c.d_y, c.d_inv, again, topk_w=c.d_w, residual=again, n_rows=c.d_n)
    assert torch.equal(out, again)
    dy, dw = c.d_y.clone(), c.empty(T, k, dtype=torch.float32)
    y, dw2 = c.d_y.clone(), c.empty(T, k, dtype=torch.float32)
    b.bqm_combine_grad(c.d_dout, c.d_inv, y=c.d_y, topk_w=c.d_w, dy=dy, dtopk_w=dw, n_rows=c.d_n)
    b.bqm_combine_grad(c.d_dout, c.d_inv, y=y, topk_w=c.d_w, dy=y, dtopk_w=dw2, n_rows=c.d_n)
    assert torch.equal(dy[:c.n], y[:c.n]) and torch.equal(dw, dw2)


def test_two_pairs_at_one_row():
    log("a place that occurs twice")
    b = _bqm()
    c = Case(6, 2, 48, "all")
    c.inv[:, 1] = c.inv[::-1, 0]
    d_inv = dev(c.inv)
    got = host(b.bqm_dispatch(c.d_x, d_inv, c.empty(c.R, 48)))
    for at in np.unique(c.inv):
        assert any((got[at] == c.x[t]).all() for t in np.argwhere(c.inv == at)[:, 0])
    ref, mag = oracle.combine(c.y, c.inv, c.R, c.w)
    out = b.bqm_combine(c.d_y, d_inv, c.empty(6, 48), topk_w=c.d_w)
    within(host(out), ref, F8 * np.abs(ref) + 7 * F24 * mag, "out")


def test_gradients_are_the_differences():
    """The combine is linear in y and in the weights: what its gradients say of a step, the
    difference of two sums of its outputs says too."""
    log("gradients against differences")
    b = _bqm()
    T, k, H = 5, 3, 16
    c = Case(T, k, H, "dropped")
    y = np.where(np.isnan(c.y), 0.0, c.y)
    rng = np.random.default_rng(5)
    step_y, step_w = bf16(rng.standard_normal(y.shape)), rng.standard_normal(c.w.shape).astype(np.float32)
    dy, dw, _ = oracle.combine_grad(c.dout, y, c.inv, c.n, c.w, np.zeros_like(y))
    import torch
    g_dy, g_dw = torch.zeros((c.R, H), dtype=torch.bfloat16, device=gpu()), c.empty(T, k, dtype=torch.float32)
    b.bqm_combine_grad(c.d_dout, c.d_inv, y=dev_bf16(y), topk_w=c.d_w, dy=g_dy, dtopk_w=g_dw, n_rows=c.d_n)

    def of(y, w):
        out, mag = oracle.combine(y, c.inv, c.n, w)
        got = host(b.bqm_combine(dev_bf16(y), c.d_inv, c.empty(T, H), topk_w=dev(np.asarray(w, dtype=np.float32)), n_rows=c.d_n))
        return (c.dout * got).sum(), (np.abs(c.dout) * (F8 * np.abs(out) + (2 * k + 3) * F24 * mag)).sum()

    zero = np.zeros_like(y)
    (f1, t1), (f0, t0) = of(step_y, c.w), of(zero, c.w)
    slope = (host(g_dy) * step_y).sum()
    assert abs((f1 - f0) - slope) <= t1 + t0 + (F8 + 2 * F24) * (np.abs(dy) * np.abs(step_y)).sum()
    (f1, t1), (f0, t0) = of(y, step_w), of(y, np.zeros_like(step_w))
    slope = (host(g_dw) * step_w).sum()
    mag = oracle.combine_grad(c.dout, y, c.inv, c.n, c.w, zero)[2]
    assert abs((f1 - f0) - slope) <= t1 + t0 + H * F24 * (mag * np.abs(step_w)).sum()


def test_rows_past_four_gigabytes():
    """600000 rows of 4096: byte and element offsets pass 32 bits."""
    import torch
    log("rows past 4 GiB")
    b = _bqm()
    T, k, H = 300000, 2, 4096
    R = T * k
    g = torch.Generator(device=gpu()).manual_seed(3)
    inv = torch.randperm(R, generator=g, device=gpu()).int()
    x = torch.randn((T, H), generator=g, device=gpu(), dtype=torch.bfloat16)
    rows = b.bqm_dispatch(x, inv, torch.zeros((R, H), dtype=torch.bfloat16, device=gpu()))
    some = torch.cat([torch.arange(0, R, 997, device=gpu()), torch.tensor([R - 1], device=gpu())])
    assert torch.equal(rows[inv.long()[some]], x[some // k])
    w = torch.rand((T, k), generator=g, device=gpu())
    out = b.bqm_combine(rows, inv, torch.empty_like(x), topk_w=w)
    t = torch.unique(some // k)
    ref = x[t].double() * w[t].double().sum(1, keepdim=True)
    assert ((out[t].double() - ref).abs() <= (F8 + 9 * F24) * ref.abs()).all()
    dw = torch.empty_like(w)
    b.bqm_combine_grad(x, inv, y=rows, topk_w=w, dy=rows, dtopk_w=dw)
    ref = x[some // k].double() * w.flatten()[some].double().unsqueeze(1)
    assert ((rows[inv.long()[some]].double() - ref).abs() <= (F8 + 2 * F24) * ref.abs()).all()
    ref = x[t].double().square().sum(1, keepdim=True)
    assert ((dw[t].double() - ref).abs() <= H * F24 * ref).all()


def test_many_short_rows():
    """More workgroups than the grid's first dimension takes, of one wave, of several tokens, and
    of the most threads."""
    import torch
    log("many tokens")
    b = _bqm()
    for T, H, values in (((1 << 22) + 5, 264, 251), ((1 << 26) + 37, 16, 251), ((1 << 22) + 5, 1009, 128)):
        inv = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=gpu())
        x = (torch.arange(T, device=gpu(), dtype=torch.int32) % values).to(torch.bfloat16).unsqueeze(1).expand(T, H).contiguous()
        rows = b.bqm_dispatch(x, inv, torch.zeros_like(x))
        assert torch.equal(rows, x.flip(0))
        assert torch.equal(b.bqm_combine(rows, inv, torch.zeros_like(x)), x)
        dw = torch.empty(T, device=gpu())
        b.bqm_combine_grad(x, inv, y=rows, dtopk_w=dw)
        assert torch.equal(dw, x[:, 0].float().square() * H)    # whole numbers below 2^24: exact
        del x, rows, inv, dw


def test_no_tokens():
    import torch
    b = _bqm()
    e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=gpu())  # noqa: E731
    inv = e(0, dtype=torch.int32)
    b.bqm_dispatch(e(0, 64), inv, e(0, 64))
    b.bqm_combine(e(0, 64), inv, e(0, 64))
    b.bqm_combine_grad(e(0, 64), inv, y=e(0, 64), dy=e(0, 64))
    torch.cuda.synchronize()


def test_binding_checks_every_tensor():
    import torch
    log("binding checks")
    b = _bqm()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=gpu())  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    inv, n = z(4, 2, dtype=i32), z(1, dtype=i32)
    calls = [(b.bqm_dispatch, [z(4, 64), inv, z(8, 64), n]),
             (b.bqm_combine, [z(8, 64), inv, z(4, 64), z(4, 2, dtype=f32), z(4, 64), n]),
             (b.bqm_combine_grad, [z(4, 64), inv, z(8, 64), z(4, 2, dtype=f32), z(8, 64), z(4, 2, dtype=f32), n])]
    for f, args in calls:
        f(*args)
        for i, t in enumerate(args):
            wide = torch.zeros(*t.shape, 2, dtype=t.dtype, device=t.device)[..., 0]
            for other in (t.to(torch.float64), wide if t.numel() > 1 else None, t.cpu(), t[1:].clone()):
                if other is None:
                    continue
                with pytest.raises((b.BQMError, ValueError)):
                    f(*args[:i], other, *args[i + 1:])
    torch.cuda.synchronize()


# more than 512 tokens, where a lane has four pairs in flight: up to four, more, and several turns of
# them; several tokens per wave, one, and rows of single elements
MANY = [(513, 1, 264), (700, 8, 264), (600, 6, 64), (520, 9, 7), (515, 5, 2080), (530, 17, 24), (1025, 4, 601), (514, 12, 33),
        (777, 7, 256), (513, 3, 8200)]


@pytest.mark.parametrize("kind", ["all", "dropped", "none"])
@pytest.mark.parametrize("T,k,H", MANY)
def test_many_tokens_against_oracle(T, k, H, kind):
    test_against_oracle(T, k, H, kind)


@pytest.mark.parametrize("T,k,H", [(600, 8, 264), (513, 6, 40), (555, 9, 601)])
def test_many_tokens_in_place(T, k, H):
    test_in_place(T, k, H)
