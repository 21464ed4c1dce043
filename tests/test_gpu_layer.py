"""The rows between token and expert order and the dense product together, as a layer uses them:
routed experts over MXFP4 beside a shared expert, on a residual stream, with a dense layer behind,
forward and backward; in a captured graph, on two streams at once, and what the binding refuses.

Tolerances as in test_gpu_linear.py and test_gpu_rows.py, for each operator on its own inputs."""
import numpy as np
import pytest

from oracle import linear as dense
from oracle import rows as order
from tests.gpu_util import gpu, log
from tests.test_gpu_linear import F8, F23, F24, eval_err, host, rounded, within

pytestmark = pytest.mark.gpu


def _bqm():
    import bit_quantized_moe_amd as bqm
    return bqm


class Layer:
    """T tokens of H to k of E experts of width I and a shared one of width S, then a dense layer of
    N; of the tokens, some are padding and some pairs go to no expert."""

    def __init__(self, T, E, k, H, I, S, N, seed=0):
        import torch
        b = _bqm()
        d = gpu()
        g = torch.Generator(device=d).manual_seed(1000 * seed + T)
        bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
        r = lambda *s, std=1.0: (torch.randn(s, generator=g, device=d) * std).to(bf)  # noqa: E731
        e = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype, device=d)  # noqa: E731
        self.T, self.E, self.k, self.H, self.I, self.S, self.N, R = T, E, k, H, I, S, N, T * k
        self.x, self.df = r(T, H), r(T, N)
        idx = torch.rand((T, E), generator=g, device=d).topk(k, 1).indices.int()
        if T > 4:
            idx[T // 2] = -1
            idx[::5, 0] = E
        self.idx, self.w = idx, torch.rand((T, k), generator=g, device=d)
        self.q_gu, self.q_dn = (b.bqm_quantize_mxfp4(r(*s, std=0.05), b.alloc_qtensor(b.FMT_MXFP4, *s))
                                for s in ((E, 2 * I, H), (E, H, I)))
        self.w_gu, self.w_dn, self.w1, self.b1 = r(2 * S, H, std=H ** -0.5), r(H, S, std=S ** -0.5), r(N, H, std=H ** -0.5), r(N)
        self.perm, self.inv, self.off = e(R, dtype=i32), e(R, dtype=i32), e(E + 1, dtype=i32)
        self.pws = e(max(16, b.bqm_permute_workspace_size(T, E, k)), dtype=u8)
        self.ws = e(max(16, *(b.bqm_linear_workspace_size(T, *s) for s in ((2 * S, H), (H, S), (N, H)))), dtype=u8)
        self.rows, self.y, self.dy, self.dxr = (e(R, H) for _ in range(4))
        self.rq, self.xq, self.aq = (b.alloc_qtensor(b.FMT_MXFP4, 1, *s) for s in ((R, H), (T, H), (R, I)))
        self.h, self.h_perm, self.h8, self.s8 = e(R, 2 * I), e(R, 2 * I), e(R, 2 * I, dtype=u8), e(R, 2 * I // 32, dtype=u8)
        self.da, self.dh = e(R, I), e(R, 2 * I)
        self.hs, self.h8s, self.s8s = e(T, 2 * S), e(T, 2 * S, dtype=u8), e(T, 2 * S // 32, dtype=u8)
        self.a, self.da_s, self.dhs = e(T, S), e(T, S), e(T, 2 * S)
        self.shared, self.out, self.z, self.f = e(T, H), e(T, H), e(T, N), e(T, N)
        self.dz, self.dout, self.dxs, self.dx = e(T, N), e(T, H), e(T, H), e(T, H)
        self.dw = e(T, k, dtype=f32)
        self.g1, self.gb1, self.g_dn, self.g_gu = (e(*s, dtype=f32) for s in ((N, H), (N,), (H, S), (2 * S, H)))

    def forward(self):
        b, n = _bqm(), self.off[self.E:]
        b.bqm_permute(self.idx, self.T, self.E, self.k, self.perm, self.inv, self.off, self.pws)
        # the experts' rows by a copy in their order, and by the product's own gather
        b.bqm_quantize_mxfp4(b.bqm_dispatch(self.x, self.inv, self.rows, n_rows=n), self.rq)
        b.bqm_mxfp4_gemm(self.rq, self.q_gu, self.off, None, 1, self.h)
        b.bqm_mxfp4_gemm(b.bqm_quantize_mxfp4(self.x, self.xq), self.q_gu, self.off, self.perm, self.k, self.h_perm)
        b.bqm_swiglu_ckpt_fwd(self.h, self.h8, self.s8, aq=self.aq, n_rows=n)
        b.bqm_mxfp4_gemm(self.aq, self.q_dn, self.off, None, 1, self.y)
        b.bqm_linear_fwd(self.x, self.w_gu, self.hs, ws=self.ws)
        b.bqm_swiglu_ckpt_fwd(self.hs, self.h8s, self.s8s, a=self.a)
        b.bqm_linear_fwd(self.a, self.w_dn, self.shared, residual=self.x, ws=self.ws)
        b.bqm_combine(self.y, self.inv, self.out, topk_w=self.w, residual=self.shared, n_rows=n)
        b.bqm_linear_fwd(self.out, self.w1, self.f, bias=self.b1, act=b.ACT_GELU_TANH, z=self.z, ws=self.ws)

    def backward(self):
        b, n = _bqm(), self.off[self.E:]
        b.bqm_act_grad(self.df, self.z, b.ACT_GELU_TANH, self.dz)
        b.bqm_linear_dgrad(self.dz, self.w1, self.dout, ws=self.ws)
        b.bqm_linear_wgrad(self.dz, self.out, self.g1, dbias=self.gb1, ws=self.ws)
        b.bqm_combine_grad(self.dout, self.inv, y=self.y, topk_w=self.w, dy=self.dy, dtopk_w=self.dw, n_rows=n)
        b.bqm_mxfp4_dgrad(self.q_dn, self.dy, self.off, None, 1, self.da)
        b.bqm_swiglu_ckpt_bwd(self.h8, self.s8, self.da, None, None, self.dh, n_rows=n)
        b.bqm_mxfp4_dgrad(self.q_gu, self.dh, self.off, None, 1, self.dxr)
        b.bqm_linear_dgrad(self.dout, self.w_dn, self.da_s, ws=self.ws)
        b.bqm_linear_wgrad(self.dout, self.a, self.g_dn, ws=self.ws)
        b.bqm_swiglu_ckpt_bwd(self.h8s, self.s8s, self.da_s, None, None, self.dhs)
        b.bqm_linear_dgrad(self.dhs, self.w_gu, self.dxs, add=self.dout, ws=self.ws)
        b.bqm_linear_wgrad(self.dhs, self.x, self.g_gu, ws=self.ws)
        b.bqm_combine(self.dxr, self.inv, self.dx, residual=self.dxs, n_rows=n)

    def step(self):
        self.forward()
        self.backward()

    NAMES = ("rows", "y", "hs", "a", "shared", "out", "z", "f", "dz", "dout", "g1", "gb1", "dy", "dw", "dxr", "da_s", "g_dn",
             "dhs", "dxs", "g_gu", "dx")

    def outputs(self):
        return {n: getattr(self, n).clone() for n in self.NAMES}

    def check(self):
        import torch
        T, k, H = self.T, self.k, self.H
        v = {n: host(getattr(self, n)) for n in self.NAMES + ("x", "df", "w_gu", "w_dn", "w1", "b1", "w")}
        inv, n = host(self.inv).astype(np.int64).reshape(T, k), int(self.off[self.E])
        assert (v["rows"] == order.dispatch(v["x"], inv, n, np.zeros_like(v["rows"]))).all()
        assert torch.equal(self.h, self.h_perm)
        for out, rows, w, res in (("out", "y", v["w"], "shared"), ("dx", "dxr", None, "dxs")):
            ref, mag = order.combine(v[rows], inv, n, w, v[res])
            within(v[out], ref, F8 * np.abs(ref) + (2 * k + 3) * F24 * mag, out)
        dy, dw, mag = order.combine_grad(v["dout"], v["y"], inv, n, v["w"], np.zeros_like(v["dy"]))
        within(v["dy"], dy, (F8 + 2 * F24) * np.abs(dy), "dy")
        within(v["dw"], dw, H * F24 * mag, "dtopk_w")
        for y, x, w, bias, name, res in (("hs", "x", "w_gu", None, "none", None), ("shared", "a", "w_dn", None, "none", "x"),
                                         ("z", "out", "w1", "b1", "none", None), ("f", "out", "w1", "b1", "gelu_tanh", None)):
            ref, z, mag = dense.fwd(v[x], v[w], None if bias is None else v[bias], name, None if res is None else v[res])
            err = (v[x].shape[1] + 1) * F23 * mag
            err = 1.13 * err + eval_err(z, name) + F23 * (np.abs(dense.act(z, name)) + np.abs(ref))
            within(v[y], ref, rounded(ref, err), y)
        ref = v["df"] * dense.act_grad(v["z"], "gelu_tanh")
        within(v["dz"], ref, rounded(ref, np.abs(v["df"]) * eval_err(v["z"], "gelu_tanh", True) + F23 * np.abs(ref)), "dz")
        for dx, dz, w, add in (("dout", "dz", "w1", None), ("da_s", "dout", "w_dn", None), ("dxs", "dhs", "w_gu", "dout")):
            ref, d, mag = dense.dgrad(v[dz], v[w], None, "none", None if add is None else v[add])
            within(v[dx], ref, rounded(ref, v[dz].shape[1] * F23 * mag + F23 * (np.abs(ref) + np.abs(d))), dx)
        for g, dz, x, gb in (("g1", "dz", "out", "gb1"), ("g_dn", "dout", "a", None), ("g_gu", "dhs", "x", None)):
            rw, mw, rb, mb = dense.wgrad(v[dz], v[x])
            within(v[g], rw, T * F23 * mw, g)
            if gb:
                within(v[gb], rb, T * F24 * mb, gb)


@pytest.mark.parametrize("T,E,k,H,I,S,N", [(1, 8, 2, 64, 32, 32, 24), (37, 16, 4, 320, 96, 128, 200), (300, 6, 2, 256, 160, 96, 520),
                                           (1200, 12, 3, 512, 64, 288, 1032)])
def test_step(T, E, k, H, I, S, N):
    log(f"layer T={T} E={E} k={k} H={H} I={I} S={S} N={N}")
    L = Layer(T, E, k, H, I, S, N)
    L.step()
    L.check()


@pytest.mark.parametrize("T", [1, 40, 1200])
def test_captured_and_replayed(T):
    """Replays between another layer's eager work, on new inputs from one to the next."""
    import torch
    log(f"layer in a graph, T={T}")
    L, other = Layer(T, 12, 3, 256, 96, 64, 264), Layer(9, 12, 3, 256, 96, 64, 264, seed=1)
    other.step()
    L.step()
    torch.cuda.synchronize()
    want_other = other.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        L.step()
    for i in range(5):
        L.x.add_(0.25)
        L.w.mul_(0.75)
        L.step()
        want = L.outputs()
        for n in L.NAMES:
            if n not in ("rows", "dy", "y", "dxr"):     # what no pair stands at is left as it was there
                getattr(L, n).zero_()
        L.ws.fill_(0xFF)
        graph.replay()
        other.step()
        torch.cuda.synchronize()
        assert all(torch.equal(v, want[n]) for n, v in L.outputs().items()), i
        assert all(torch.equal(v, want_other[n]) for n, v in other.outputs().items()), i


def test_two_streams_at_once():
    import torch
    log("two layers on two streams")
    a, b = Layer(1100, 10, 2, 512, 64, 96, 1032), Layer(45, 10, 2, 192, 64, 96, 136, seed=3)
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


def test_a_stream_given_as_an_argument():
    import torch
    log("a stream as an argument")
    b, d = _bqm(), gpu()
    g = torch.Generator(device=d).manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device=d).bfloat16()  # noqa: E731
    x, w, dz = r(300, 136), r(264, 136), r(300, 264)
    inv = torch.randperm(600, generator=g, device=d).int()
    rows, tw = r(600, 136), torch.rand((300, 2), generator=g, device=d)
    ws = torch.zeros(max(16, b.bqm_linear_workspace_size(300, 264, 136)), dtype=torch.uint8, device=d)

    def run(stream):
        o = [torch.zeros_like(t) for t in (rows, x, rows, dz, x, dz)] + [torch.zeros((264, 136), device=d), torch.zeros(264, device=d)]
        torch.cuda.synchronize()
        b.bqm_dispatch(x, inv, o[0], stream=stream)
        b.bqm_combine(rows, inv, o[1], topk_w=tw, stream=stream)
        b.bqm_combine_grad(x, inv, topk_w=tw, dy=o[2], stream=stream)
        b.bqm_linear_fwd(x, w, o[3], ws=ws, stream=stream)
        b.bqm_linear_dgrad(dz, w, o[4], ws=ws, stream=stream)
        b.bqm_act_grad(dz, dz, b.ACT_SILU, o[5], stream=stream)
        b.bqm_linear_wgrad(dz, x, o[6], dbias=o[7], ws=ws, stream=stream)
        torch.cuda.synchronize()
        return o
    assert all(torch.equal(p, q) for p, q in zip(run(None), run(torch.cuda.Stream().cuda_stream)))


def test_refusals_of_the_binding(monkeypatch):
    """Host workspaces, and tensors that are not on the current device."""
    import torch
    log("binding, device checks")
    b = _bqm()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=gpu())  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    x, w, y = z(4, 64), z(16, 64), z(4, 16)
    rows, inv = z(8, 64), z(8, dtype=i32)
    calls = [lambda ws: b.bqm_linear_fwd(x, w, y, ws=ws), lambda ws: b.bqm_linear_dgrad(y, w, x, ws=ws),
             lambda ws: b.bqm_linear_wgrad(y, x, z(16, 64, dtype=f32), ws=ws)]
    for f in calls:
        with pytest.raises(b.BQMError, match="ws: not a GPU tensor"):
            f(torch.zeros(1 << 16, dtype=torch.uint8))
        with pytest.raises(b.BQMError, match="ws: not contiguous"):
            f(z(1 << 17, dtype=torch.uint8)[::2])
        with pytest.raises(b.BQMError, match="ws: dtype"):
            f(z(1 << 14, dtype=f32))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: x.get_device() + 1)
    for f in [lambda f=f: f(None) for f in calls] + [lambda: b.bqm_dispatch(x, inv, rows), lambda: b.bqm_combine(rows, inv, x),
                                                     lambda: b.bqm_combine_grad(x, inv, dy=rows), lambda: b.bqm_act_grad(y, y, 1, y)]:
        with pytest.raises(b.BQMError, match="on device"):
            f()
