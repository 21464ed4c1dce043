"""Argument checks of the dense product's entry points (host only: every call here fails, or is
empty, before anything is launched)."""
import pytest

torch = pytest.importorskip("torch")
bqm = pytest.importorskip("bit_quantized_moe_amd._lib")


@pytest.fixture(scope="module")
def lib():
    return bqm.load()


def sizes(f):
    assert f(M=-1) == -1 and f(M=1 << 30) == -2 and f(M=1 << 31) == -2
    assert f(N=0) == -2 and f(N=12) == -2 and f(N=-8) == -2 and f(N=1 << 22) == -2
    assert f(K=0) == -2 and f(K=4) == -2 and f(K=1 << 22) == -2 and "K=" in bqm.bqm_last_error()
    assert f(M=(1 << 30) - 1, N=(1 << 22) - 8) == -2 and "tiles" in bqm.bqm_last_error()


def test_forward(lib):
    def f(x=16, w=16, bias=16, act=0, res=16, M=4, N=64, K=64, y=16, z=16, ws=16, wsb=1 << 30):
        return lib.bqm_linear_fwd(x, w, bias, act, res, M, N, K, y, z, ws, wsb, None)
    sizes(f)
    assert f(act=-1) == -1 and f(act=4) == -1
    assert f(x=None) == -1 and f(w=None) == -1 and f(y=None) == -1
    for name in ("x", "w", "bias", "res", "y", "z"):
        assert f(**{name: 24}) == -3, name
    assert f(M=0, x=None, w=None, y=None, ws=None) == 0


def test_input_gradient(lib):
    def f(dz=16, w=16, zx=16, act=1, add=16, M=4, N=64, K=64, dx=16, ws=16, wsb=1 << 30):
        return lib.bqm_linear_dgrad(dz, w, zx, act, add, M, N, K, dx, ws, wsb, None)
    sizes(f)
    assert f(act=-1) == -1 and f(act=4) == -1
    assert f(dz=None) == -1 and f(w=None) == -1 and f(dx=None) == -1
    assert f(zx=None) == -1 and "needs zx" in bqm.bqm_last_error()
    for name in ("dz", "w", "zx", "add", "dx"):
        assert f(**{name: 24}) == -3, name
    assert f(M=0, dz=None, w=None, zx=None, dx=None, ws=None) == 0


def test_weight_gradient(lib):
    def f(dz=16, x=16, acc=0, M=4, N=64, K=64, dw=16, db=16, ws=16, wsb=1 << 30):
        return lib.bqm_linear_wgrad(dz, x, acc, M, N, K, dw, db, ws, wsb, None)
    sizes(f)
    assert f(dz=None) == -1 and f(x=None) == -1 and f(dw=None) == -1
    for name in ("dz", "x", "dw", "db"):
        assert f(**{name: 24}) == -3, name
    assert f(M=0, acc=1, dz=None, x=None) == 0      # nothing to add
    assert f(M=0, acc=1, dw=None) == -1


def test_act_grad(lib):
    def f(dy=16, z=16, act=2, n=64, dz=16):
        return lib.bqm_act_grad(dy, z, act, n, dz, None)
    assert f(act=0) == -1 and f(act=4) == -1 and f(act=-2) == -1
    assert f(n=-1) == -1 and f(n=1 << 34) == -2
    assert f(dy=None) == -1 and f(z=None) == -1 and f(dz=None) == -1
    assert f(dy=8) == -3 and f(z=8) == -3 and f(dz=8) == -3
    assert f(n=0, dy=None, z=None, dz=None) == 0


# the weight gradient of many rows splits its contraction, or its bias gradient's
@pytest.mark.parametrize("M,N,K", [(16384, 4096, 6144), (8192, 264, 264), (100000, 64, 64)])
def test_workspace(lib, M, N, K):
    n = lib.bqm_linear_workspace_size(M, N, K)
    assert 0 < n <= (72 << 20) and n % 256 == 0
    for ws, wsb in ((None, 1 << 30), (16, 0), (16, 1024)):
        assert lib.bqm_linear_wgrad(16, 16, 0, M, N, K, 16, 16, ws, wsb, None) == -5
    assert lib.bqm_linear_wgrad(16, 16, 0, M, N, K, 16, 16, 24, 1 << 30, None) == -3


def test_workspace_of_what_needs_none(lib):
    assert lib.bqm_linear_workspace_size(0, 64, 64) == 0
    assert lib.bqm_linear_workspace_size(-1, 64, 64) == 0 and lib.bqm_linear_workspace_size(4, 60, 64) == 0
    assert lib.bqm_linear_workspace_size(4, 8, 8) == 0


def test_binding():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    f32 = torch.float32
    bad = [
        ("x: dtype", lambda: bqm.bqm_linear_fwd(z(4, 64, dtype=f32), z(16, 64), z(4, 16))),
        ("x: not contiguous", lambda: bqm.bqm_linear_fwd(z(64, 4).t(), z(16, 64), z(4, 16))),
        ("not a GPU tensor", lambda: bqm.bqm_linear_fwd(z(4, 64), z(16, 64), z(4, 16))),
        ("dz: shape", lambda: bqm.bqm_linear_dgrad(z(4, 24), z(16, 64), z(4, 64))),
        ("dz: dtype", lambda: bqm.bqm_linear_wgrad(z(4, 16, dtype=torch.float16), z(4, 64), z(16, 64, dtype=f32))),
        ("dy: dtype", lambda: bqm.bqm_act_grad(z(4, dtype=f32), z(4), 1, z(4))),
    ]
    for what, f in bad:
        with pytest.raises(bqm.BQMError, match=what):
            f()
