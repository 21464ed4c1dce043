"""Argument checks of the entry points for rows between token order and expert order (host
only: every call here fails, or is empty, before anything is launched)."""
import pytest

torch = pytest.importorskip("torch")
bqm = pytest.importorskip("bit_quantized_moe_amd._lib")


@pytest.fixture(scope="module")
def lib():
    return bqm.load()


def sizes(f):
    """What the three calls ask of T, H, k and the places."""
    assert f(T=-1) == -1
    assert f(k=0) == -2 and f(k=-3) == -2
    assert f(H=0) == -2 and f(H=-8) == -2 and f(H=1 << 24) == -2
    assert f(T=1 << 31) == -2 and f(T=1 << 30, k=2) == -2 and f(T=(1 << 62) + 1, k=4) == -2
    assert f(inv=None) == -1 and f(inv=18) == -3 and f(n=18) == -3


def test_dispatch(lib):
    def f(x=16, inv=16, T=4, H=64, k=2, n=None, rows=16):
        return lib.bqm_dispatch(x, inv, T, H, k, n, rows, None)
    sizes(f)
    assert f(x=None) == -1 and f(rows=None) == -1 and "NULL" in bqm.bqm_last_error()
    assert f(x=24) == -3 and f(rows=8) == -3
    assert f(T=0, x=None, inv=None, rows=None) == 0


def test_combine(lib):
    def f(y=16, inv=16, w=16, res=None, T=4, H=64, k=2, n=None, out=16):
        return lib.bqm_combine(y, inv, w, res, T, H, k, n, out, None)
    sizes(f)
    assert f(y=None) == -1 and f(out=None) == -1
    assert f(y=8) == -3 and f(w=4) == -3 and f(res=2) == -3 and f(out=24) == -3
    assert f(T=0, y=None, inv=None, out=None) == 0


def test_combine_grad(lib):
    def f(dout=16, y=16, inv=16, w=16, T=4, H=64, k=2, n=None, dy=16, dw=16):
        return lib.bqm_combine_grad(dout, y, inv, w, T, H, k, n, dy, dw, None)
    sizes(f)
    assert f(dout=None) == -1 and f(y=None) == -1 and "needs y" in bqm.bqm_last_error()
    assert f(dy=None, dw=None) == -1 and "both" in bqm.bqm_last_error()
    assert f(dout=8) == -3 and f(y=8) == -3 and f(w=8) == -3 and f(dy=8) == -3 and f(dw=8) == -3
    assert f(T=0, dout=None, y=None, inv=None) == 0


def test_binding():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    inv = z(4, 2, dtype=i32)
    bad = [
        ("inv: 7 pairs for 4 tokens", lambda: bqm.bqm_dispatch(z(4, 64), z(7, dtype=i32), z(7, 64))),
        ("inv: 8 pairs for 0 tokens", lambda: bqm.bqm_combine(z(8, 64), inv, z(0, 64))),
        ("inv: 0 pairs for 4 tokens", lambda: bqm.bqm_combine_grad(z(4, 64), z(0, dtype=i32), z(0, 64), dy=z(0, 64))),
        ("x: dtype", lambda: bqm.bqm_dispatch(z(4, 64, dtype=f32), inv, z(8, 64))),
        ("x: not contiguous", lambda: bqm.bqm_dispatch(z(64, 4).t(), inv, z(8, 64))),
        ("not a GPU tensor", lambda: bqm.bqm_dispatch(z(4, 64), inv, z(8, 64))),
        ("y: shape", lambda: bqm.bqm_combine(z(7, 64), inv, z(4, 64))),
        ("y: dtype", lambda: bqm.bqm_combine(z(8, 64, dtype=torch.float16), inv, z(4, 64))),
        ("dout: dtype", lambda: bqm.bqm_combine_grad(z(4, 64, dtype=f32), inv, dy=z(8, 64))),
    ]
    for what, f in bad:
        with pytest.raises(bqm.BQMError, match=what):
            f()
