"""Argument checks of the MXFP4 expert and router entry points (host only: every call here
fails, or is empty, before anything is launched)."""
import ctypes as C
import sys

import pytest

torch = pytest.importorskip("torch")
bqm = pytest.importorskip("bit_quantized_moe_amd._lib")


@pytest.fixture(scope="module")
def lib():
    return bqm.load()


def q(n=1, rows=64, cols=64, fmt=3, codes=16, scales=16):
    return bqm.QTensorC(fmt, 0, n, rows, cols, codes, scales, None, 1, 0)


def test_quantize_mxfp4(lib):
    f = lib.bqm_quantize_mxfp4
    assert f(16, C.byref(q(cols=48)), None) == -2 and "multiple of 32" in bqm.bqm_last_error()
    assert f(16, C.byref(q(fmt=1)), None) == -1
    assert f(16, C.byref(q(fmt=4)), None) == -1
    assert f(None, C.byref(q()), None) == -1
    assert f(24, C.byref(q()), None) == -3
    assert f(16, C.byref(q(codes=None)), None) == -1
    assert f(16, C.byref(q(scales=8)), None) == -3
    assert f(16, C.byref(q(rows=-1)), None) == -1
    assert f(None, C.byref(q(rows=0)), None) == 0
    assert f(16, None, None) == -1
    # the other quantizers and the layer do not take the format
    assert lib.bqm_quantize_nvfp4(16, 1, None, C.byref(q()), 16, 64, None) == -1
    assert lib.bqm_quantize_nf4(16, C.byref(q()), None) == -1
    nested = q()
    nested.nested = 1
    assert lib.bqm_dequantize(C.byref(nested), 16, None) == -1
    d = bqm.MoEDescC(64, 64, 64, 1, 1, 0, 0, 1.0, 0, q(rows=128), q(), None, None, None, None, None)
    assert lib.bqm_moe_fwd(C.byref(d), 16, 16, 16, 16, 16, 1 << 40, None) == -1


def test_gemm(lib):
    def f(x=None, w=None, off=16, perm=None, k=1, R=64, y=16):
        return lib.bqm_mxfp4_gemm(C.byref(x or q()), C.byref(w or q(n=4)), off, perm, k, R, y, None)
    assert f(x=q(fmt=1)) == -1 and f(w=q(n=4, fmt=2)) == -1
    assert f(x=q(n=2)) == -2                           # x is one matrix
    assert f(x=q(cols=96)) == -2                       # K differs
    assert f(x=q(cols=48), w=q(n=4, cols=48)) == -2    # K % 32
    assert f(w=q(n=4, rows=40)) == -2                  # N % 32
    assert f(w=q(n=4, rows=0)) == -2 and f(w=q(n=0)) == -2 and f(w=q(n=1025)) == -2
    assert f(R=63) == -2                               # rows without perm
    assert f(perm=16, k=2, R=127) == -2 and f(perm=16, k=0, R=64) == -2
    assert f(R=-1) == -1
    assert f(x=q(rows=1 << 62), perm=16, k=4, R=0) == -2   # rows k = 0 in 64 bits
    assert f(off=None) == -1 and f(off=20) == -3 and f(perm=20) == -3
    assert f(y=None) == -1 and f(y=20) == -3
    assert f(x=q(codes=None)) == -1 and f(w=q(n=4, scales=18)) == -3
    assert lib.bqm_mxfp4_gemm(None, C.byref(q()), 16, None, 1, 64, 16, None) == -1
    assert f(x=q(rows=1 << 30), R=1 << 30) == -2
    assert f(x=q(rows=0, codes=None, scales=None), R=0, off=None, y=None) == 0


def test_dgrad(lib):
    def f(w=None, dy=16, rows=64, off=16, perm=None, k=1, R=64, dx=16):
        return lib.bqm_mxfp4_dgrad(C.byref(w or q(n=4)), dy, rows, off, perm, k, R, dx, None)
    assert f(w=q(fmt=1)) == -1 and f(w=q(rows=33)) == -2 and f(w=q(cols=33)) == -2
    assert f(rows=63) == -2 and f(perm=16, k=3, R=64) == -2 and f(rows=-1, R=-1) == -1
    assert f(dy=None) == -1 and f(dx=None) == -1 and f(dy=17) == -3 and f(dx=18) == -3
    assert f(off=None) == -1
    assert f(rows=0, R=0, dy=None, dx=None, off=None) == 0


def test_swiglu(lib):
    def f(h=16, R=4, I=64, h8=16, s=16, a=16, aq=None):
        return lib.bqm_swiglu_ckpt_fwd(h, R, I, None, h8, s, a, None if aq is None else C.byref(aq), None)
    assert f(I=48) == -2 and f(I=0) == -2 and f(R=-1) == -1 and f(R=1 << 31) == -2
    assert f(h=None) == -1 and f(h8=None) == -1 and f(s=None) == -1
    assert f(h=8) == -3 and f(h8=8) == -3 and f(s=8) == -3 and f(a=8) == -3
    assert f(aq=q(rows=4, fmt=1)) == -1 and f(aq=q(rows=5)) == -2 and f(aq=q(rows=4, codes=None)) == -1
    assert f(aq=q(rows=4, scales=20)) == -3
    assert f(R=0, h=None, h8=None, s=None, a=None) == 0

    def g(h8=16, s=16, da=16, perm=16, w=16, R=4, I=64, dh=16, dw=16):
        return lib.bqm_swiglu_ckpt_bwd(h8, s, da, perm, w, R, I, None, dh, dw, None)
    assert g(I=16) == -2 and g(R=-2) == -1 and g(da=None) == -1 and g(dh=None) == -1 and g(h8=None) == -1
    assert g(perm=4) == -3 and g(w=4) == -3 and g(dw=4) == -3 and g(dh=4) == -3
    assert g(R=0, h8=None, s=None, da=None, dh=None) == 0


def test_router(lib):
    def f(l=16, idx=16, valid=None, T=4, E=8, k=2, counts=16, loss=16, ws=16, wsb=1 << 30):
        return lib.bqm_router_loss(l, idx, valid, T, E, k, counts, loss, ws, wsb, None)
    assert f(E=0) == -2 and f(E=1025) == -2 and f(k=9) == -2 and f(k=0) == -2 and f(E=64, k=17) == -2
    assert f(T=-1) == -1 and f(T=1 << 30) == -2 and f(T=1 << 62, k=4) == -2   # T k = 0 in 64 bits
    assert f(l=None) == -1 and f(idx=None) == -1 and f(counts=None) == -1 and f(loss=None) == -1
    assert f(l=8) == -3 and f(valid=8) == -3 and f(loss=8) == -3 and f(ws=8) == -3
    assert f(ws=None) == -5 and f(wsb=lib.bqm_router_loss_workspace_size(4, 8) - 1) == -5
    assert lib.bqm_router_loss_workspace_size(-1, 8) == 0 and lib.bqm_router_loss_workspace_size(4, 0) == 0
    assert lib.bqm_router_loss_workspace_size(1 << 20, 1024) >= lib.bqm_router_loss_workspace_size(1, 1024) > 0

    def g(l=16, idx=16, valid=None, counts=16, dw=None, dl=None, T=4, E=8, k=2, out=16):
        return lib.bqm_router_grad(l, idx, valid, counts, dw, dl, T, E, k, 0, out, None)
    assert g(E=2000) == -2 and g(k=9) == -2 and g(T=-1) == -1
    assert g(l=None) == -1 and g(idx=None) == -1 and g(counts=None) == -1 and g(out=None) == -1
    assert g(dw=8) == -3 and g(dl=8) == -3 and g(out=8) == -3
    assert g(T=0, l=None, idx=None, counts=None, out=None) == 0


def test_binding_checks_types_shapes_and_layout():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    mxq = lambda n, r, c: bqm.alloc_qtensor(bqm.FMT_MXFP4, n, r, c, device="cpu")  # noqa: E731
    off, w, x = z(5, dtype=torch.int32), mxq(4, 64, 32), mxq(1, 8, 32)
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    bad = [
        ("x: dtype", lambda: bqm.bqm_quantize_mxfp4(z(1, 8, 32, dtype=f32), x)),
        ("x: not contiguous", lambda: bqm.bqm_quantize_mxfp4(z(1, 32, 8).transpose(1, 2), x)),
        ("x: shape", lambda: bqm.bqm_quantize_mxfp4(z(1, 8, 64), x)),
        ("x: not a GPU tensor", lambda: bqm.bqm_quantize_mxfp4(z(1, 8, 32), x)),
        ("w: format", lambda: bqm.bqm_mxfp4_dgrad(bqm.alloc_qtensor(bqm.FMT_NF4, 4, 64, 64, device="cpu"), z(8, 64), off,
                                                  None, 1, z(8, 64))),
        ("not a GPU tensor", lambda: bqm.bqm_mxfp4_gemm(x, w, off, None, 1, z(8, 64))),
        ("h: dtype", lambda: bqm.bqm_swiglu_ckpt_fwd(z(4, 128, dtype=f32), z(4, 128, dtype=u8), z(4, 4, dtype=u8))),
        ("h: not contiguous", lambda: bqm.bqm_swiglu_ckpt_fwd(z(128, 4).t(), z(4, 128, dtype=u8), z(4, 4, dtype=u8))),
        ("h8: shape", lambda: bqm.bqm_swiglu_ckpt_bwd(z(4, 64, dtype=u8), z(4, 4, dtype=u8), z(4, 64), None, None,
                                                      z(4, 128))),
        ("h8: dtype", lambda: bqm.bqm_swiglu_ckpt_bwd(z(4, 128), z(4, 4, dtype=u8), z(4, 64), None, None, z(4, 128))),
        ("logits: dtype", lambda: bqm.bqm_router_grad(z(4, 8), z(4, 2, dtype=i32), None, z(9, dtype=i32), None, None, 0,
                                                      z(4, 8, dtype=f32))),
        ("logits: not contiguous", lambda: bqm.bqm_router_loss(z(8, 4, dtype=f32).t(), z(4, 2, dtype=i32), None,
                                                               z(9, dtype=i32), z(2, dtype=f32), None)),
    ]
    for what, f in bad:
        with pytest.raises(bqm.BQMError, match=what):
            f()


def test_dequantize_of_mxfp4_checks_its_tensors(monkeypatch):
    """An output of another size, type or layout, or codes of another size, are refused before
    anything is launched."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    q = bqm.alloc_qtensor(bqm.FMT_MXFP4, 2, 8, 64, device="cpu")
    short = bqm.alloc_qtensor(bqm.FMT_MXFP4, 2, 8, 64, device="cpu")
    short.codes = short.codes[:1].clone()
    few = bqm.alloc_qtensor(bqm.FMT_MXFP4, 2, 8, 64, device="cpu")
    few.scales = few.scales[..., :1].clone()
    with pytest.raises(bqm.BQMError, match="not a GPU tensor"):
        bqm.bqm_dequantize(q, z(2, 8, 64))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)    # host tensors pass the device check
    for what, f in [
        ("y: shape", lambda: bqm.bqm_dequantize(q, z(1, 8, 64))),
        ("y: dtype", lambda: bqm.bqm_dequantize(q, z(2, 8, 64, dtype=torch.float32))),
        ("y: not contiguous", lambda: bqm.bqm_dequantize(q, z(2, 64, 8).transpose(1, 2))),
        ("codes: shape", lambda: bqm.bqm_dequantize(short, z(2, 8, 64))),
        ("scales: shape", lambda: bqm.bqm_dequantize(few, z(2, 8, 64))),
    ]:
        with pytest.raises(bqm.BQMError, match=what):
            f()


@pytest.mark.parametrize("E", [1, 8, 16, 17, 32, 33, 64, 128, 256, 1024])
def test_router_loss_workspace_has_no_part_without_tokens(lib, E):
    """A part of the workspace holds E sums and E counts of 4 bytes for a workgroup of the
    first kernel; a workgroup of 1024 threads takes 1024 / lanes tokens at a time, and there
    are no more of them than get any.  (Arrays are padded to 256 bytes.)"""
    lanes = 4 if E <= 16 else 8 if E <= 32 else 16 if E <= 64 else 32 if E <= 128 else 64
    for T in (1, 2049, 4096, 5000, 65536, 1 << 20):
        parts = -(-T // (1024 // lanes))
        most = 2 * (parts * E * 4 + 255) + 2 * (parts * 4 + 255) + 2 * 256
        assert lib.bqm_router_loss_workspace_size(T, E) <= most, T


def test_binding_without_torch_s_private_calls(lib, monkeypatch):
    """The current stream and device through torch's public interface, where the private calls
    that the binding takes them from are not there."""
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("Stream", (), {"cuda_stream": 77})())
    assert bqm._stream(None) == 77 and bqm._stream(5) == 5
    assert bqm._begin() == (lib, 3)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    assert bqm._begin() == (lib, -2)


def test_first_calls_of_two_threads_at_once(lib, monkeypatch):
    """Wherever another thread's first call comes between two instructions of this one's, it
    finds the types that its checks compare with, or sets them itself."""
    names = ("_bf16", "_f32", "_i32", "_u8")
    for name in ("_torch", *names):
        monkeypatch.setattr(bqm, name, None)
    half = []

    def trace(frame, event, arg):
        if frame.f_code is not bqm._begin.__code__:
            return None
        frame.f_trace_opcodes = True
        if bqm._torch is not None and any(getattr(bqm, n) is None for n in names):
            half.append(frame.f_lasti)
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        bqm._begin()
    finally:
        sys.settrace(before)
    assert bqm._torch is torch and not half
