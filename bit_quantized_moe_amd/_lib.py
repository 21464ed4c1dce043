"""ctypes binding of libbqm.so: one Python function per C entry point, same names.

Only argument marshalling happens here (tensor -> device pointer, sizes, stream
handle, status -> exception); every step of the path runs in the HIP library.
torch supplies device memory and streams.  The library must be built (python -m
bit_quantized_moe_amd.build); without it every call raises.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbqm.so")

FMT_NVFP4 = 1
FMT_NF4 = 2
FMT_MXFP4 = 3
SCALE_PER_TENSOR = 0
SCALE_PER_ROW = 1
ACT_NONE = 0
ACT_RELU = 1
ACT_SILU = 2
ACT_GELU_TANH = 3

STAGES = ["permute", "act_quant_x", "lora_a_gu", "gate_up_fwd", "act_quant_a", "lora_a_dn", "down_fwd",
          "combine_fwd", "dtopk", "lora_b_dn", "down_dgrad", "lora_b_gu", "gate_up_dgrad", "combine_dgrad",
          "lora_grad"]
STAGE_COUNT = len(STAGES)

STATUS = {0: "BQM_OK", -1: "BQM_ERR_INVALID_ARG", -2: "BQM_ERR_SHAPE", -3: "BQM_ERR_ALIGN",
          -4: "BQM_ERR_UNSUPPORTED", -5: "BQM_ERR_WORKSPACE", -6: "BQM_ERR_HIP"}

EXPORTS = ["bqm_abi_version", "bqm_last_error", "bqm_quantize_nvfp4_workspace_size",
           "bqm_quantize_nvfp4", "bqm_quantize_nvfp4_noalloc", "bqm_quantize_nf4", "bqm_dequantize", "bqm_route",
           "bqm_permute_workspace_size", "bqm_permute", "bqm_moe_workspace_size", "bqm_moe_fwd",
           "bqm_moe_dgrad", "bqm_moe_dgrad_colwise", "bqm_lora_grad", "bqm_nf4_nest", "bqm_quantize_mxfp4",
           "bqm_mxfp4_gemm", "bqm_mxfp4_dgrad", "bqm_swiglu_ckpt_fwd", "bqm_swiglu_ckpt_bwd",
           "bqm_router_loss_workspace_size", "bqm_router_loss", "bqm_router_grad", "bqm_dispatch", "bqm_combine",
           "bqm_combine_grad", "bqm_linear_workspace_size", "bqm_linear_fwd", "bqm_linear_dgrad", "bqm_linear_wgrad",
           "bqm_act_grad"]


class BQMError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class QTensorC(C.Structure):
    _fields_ = [("fmt", C.c_int32), ("scale_mode", C.c_int32), ("n_mat", C.c_int64),
                ("rows", C.c_int64), ("cols", C.c_int64), ("codes", C.c_void_p),
                ("scales", C.c_void_p), ("s_dec", C.c_void_p), ("four_over_six", C.c_int32),
                ("nested", C.c_int32)]


class MoEDescC(C.Structure):
    _fields_ = [("T", C.c_int64), ("H", C.c_int64), ("I", C.c_int64), ("E", C.c_int32),
                ("k", C.c_int32), ("r", C.c_int32), ("act_quant", C.c_int32),
                ("lora_scale", C.c_float), ("lora_shared_a", C.c_int32), ("w_gu", QTensorC),
                ("w_dn", QTensorC), ("A_gu", C.c_void_p), ("B_gu", C.c_void_p),
                ("A_dn", C.c_void_p), ("B_dn", C.c_void_p), ("stage_events", C.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libbqm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with python -m bit_quantized_moe_amd.build")
    # torch first, so that the library binds to the HIP runtime torch already uses
    # (same soname: one runtime per process, shared streams and allocations)
    import torch  # noqa: F401
    lib = C.CDLL(path)
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    sig = {
        "bqm_abi_version": (C.c_int, []),
        "bqm_last_error": (C.c_char_p, []),
        "bqm_quantize_nvfp4_workspace_size": (sz, [i64, i64, i64, i32]),
        "bqm_quantize_nvfp4": (C.c_int, [vp, i32, vp, C.POINTER(QTensorC), vp, sz, vp]),
        "bqm_quantize_nvfp4_noalloc": (C.c_int, [vp, i32, vp, C.POINTER(QTensorC), vp]),
        "bqm_quantize_nf4": (C.c_int, [vp, C.POINTER(QTensorC), vp]),
        "bqm_nf4_nest": (C.c_int, [C.POINTER(QTensorC), C.POINTER(QTensorC), vp]),
        "bqm_dequantize": (C.c_int, [C.POINTER(QTensorC), vp, vp]),
        "bqm_route": (C.c_int, [vp, i64, i32, i32, i32, vp, vp, vp]),
        "bqm_permute_workspace_size": (sz, [i64, i32, i32]),
        "bqm_permute": (C.c_int, [vp, i64, i32, i32, vp, vp, vp, vp, sz, vp]),
        "bqm_moe_workspace_size": (sz, [C.POINTER(MoEDescC)]),
        "bqm_moe_fwd": (C.c_int, [C.POINTER(MoEDescC), vp, vp, vp, vp, vp, sz, vp]),
        "bqm_moe_dgrad": (C.c_int, [C.POINTER(MoEDescC), vp, vp, sz, vp, vp, vp]),
        "bqm_moe_dgrad_colwise": (C.c_int, [C.POINTER(MoEDescC), C.POINTER(QTensorC), C.POINTER(QTensorC), vp, vp,
                                            sz, vp, vp, vp]),
        "bqm_lora_grad": (C.c_int, [C.POINTER(MoEDescC), vp, vp, vp, sz, vp, vp, vp, vp, vp]),
        "bqm_quantize_mxfp4": (C.c_int, [vp, C.POINTER(QTensorC), vp]),
        "bqm_mxfp4_gemm": (C.c_int, [C.POINTER(QTensorC), C.POINTER(QTensorC), vp, vp, i32, i64, vp, vp]),
        "bqm_mxfp4_dgrad": (C.c_int, [C.POINTER(QTensorC), vp, i64, vp, vp, i32, i64, vp, vp]),
        "bqm_swiglu_ckpt_fwd": (C.c_int, [vp, i64, i64, vp, vp, vp, vp, C.POINTER(QTensorC), vp]),
        "bqm_swiglu_ckpt_bwd": (C.c_int, [vp, vp, vp, vp, vp, i64, i64, vp, vp, vp, vp]),
        "bqm_router_loss_workspace_size": (sz, [i64, i32]),
        "bqm_router_loss": (C.c_int, [vp, vp, vp, i64, i32, i32, vp, vp, vp, sz, vp]),
        "bqm_router_grad": (C.c_int, [vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, vp, vp]),
        "bqm_dispatch": (C.c_int, [vp, vp, i64, i64, i32, vp, vp, vp]),
        "bqm_combine": (C.c_int, [vp, vp, vp, vp, i64, i64, i32, vp, vp, vp]),
        "bqm_combine_grad": (C.c_int, [vp, vp, vp, vp, i64, i64, i32, vp, vp, vp, vp]),
        "bqm_linear_workspace_size": (sz, [i64, i64, i64]),
        "bqm_linear_fwd": (C.c_int, [vp, vp, vp, i32, vp, i64, i64, i64, vp, vp, vp, sz, vp]),
        "bqm_linear_dgrad": (C.c_int, [vp, vp, vp, i32, vp, i64, i64, i64, vp, vp, sz, vp]),
        "bqm_linear_wgrad": (C.c_int, [vp, vp, i32, i64, i64, i64, vp, vp, vp, sz, vp]),
        "bqm_act_grad": (C.c_int, [vp, vp, i32, i64, vp, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        msg = _lib.bqm_last_error().decode(errors="replace")
        raise BQMError(status, msg)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        try:
            # the current stream's handle without building a Stream object (0.1 us, not 2.8 us)
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:      # not part of torch's public interface
            return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


@dataclass
class QTensor:
    """A rowwise-quantized stack held in torch tensors (see bqm_qtensor)."""
    fmt: int
    scale_mode: int
    n_mat: int
    rows: int
    cols: int
    codes: object
    scales: object
    s_dec: object = None
    four_over_six: int = 1
    nested: int = 0          # NF4: 1 = double-quantized absmax (see bqm_nf4_nest)

    def c(self) -> QTensorC:
        return QTensorC(self.fmt, self.scale_mode, self.n_mat, self.rows, self.cols, _ptr(self.codes),
                        _ptr(self.scales), _ptr(self.s_dec), self.four_over_six, int(self.nested))


def nf4_nest_groups(rows, cols) -> int:
    """Groups of 256 absmax blocks per matrix of a nested NF4 stack."""
    return -(-(rows * cols // 64) // 256)


def alloc_qtensor(fmt, n_mat, rows, cols, device="cuda", scale_mode=SCALE_PER_TENSOR,
                  four_over_six=1, nested=0) -> QTensor:
    import torch
    codes = torch.empty((n_mat, rows, cols // 2), dtype=torch.uint8, device=device)
    if fmt == FMT_NVFP4:
        scales = torch.empty((n_mat, rows, cols // 16), dtype=torch.uint8, device=device)
        n = n_mat if scale_mode == SCALE_PER_TENSOR else n_mat * rows
        s_dec = torch.empty((max(n, 1),), dtype=torch.float32, device=device)
    elif fmt == FMT_MXFP4:
        scales = torch.empty((n_mat, rows, cols // 32), dtype=torch.uint8, device=device)
        s_dec = None
    elif nested:
        scales = torch.empty((n_mat, rows, cols // 64), dtype=torch.uint8, device=device)
        s_dec = torch.empty((max(n_mat, 1), 1 + nf4_nest_groups(rows, cols)), dtype=torch.float32, device=device)
    else:
        scales = torch.empty((n_mat, rows, cols // 64), dtype=torch.float32, device=device)
        s_dec = None
    return QTensor(fmt, scale_mode, n_mat, rows, cols, codes, scales, s_dec, four_over_six, nested)


def quantize_stack(w, fmt: str, stream=None) -> QTensor:
    """Allocate and fill a rowwise-quantized stack from a bf16 [n_mat, rows, cols] tensor:
    fmt "nvfp4" (per-tensor scale, Four-Over-Six), "mxfp4", "nf4" or "nf4_nested" (NF4,
    then bqm_nf4_nest; the nested stack keeps the plain codes).  Allocation plus the library
    calls, nothing else."""
    import torch
    n_mat, rows, cols = w.shape
    if fmt == "nvfp4":
        q = alloc_qtensor(FMT_NVFP4, n_mat, rows, cols, device=w.device)
        wsb = bqm_quantize_nvfp4_workspace_size(n_mat, rows, cols, SCALE_PER_TENSOR)
        ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=w.device)
        bqm_quantize_nvfp4(w, 1, None, q, ws, stream)
        return q
    if fmt == "mxfp4":
        return bqm_quantize_mxfp4(w, alloc_qtensor(FMT_MXFP4, n_mat, rows, cols, device=w.device), stream)
    if fmt not in ("nf4", "nf4_nested"):
        raise ValueError(f"unknown weight format {fmt!r}")
    q = alloc_qtensor(FMT_NF4, n_mat, rows, cols, device=w.device)
    bqm_quantize_nf4(w, q, stream)
    if fmt == "nf4":
        return q
    n = alloc_qtensor(FMT_NF4, n_mat, rows, cols, device=w.device, nested=1)
    n.codes = q.codes
    bqm_nf4_nest(q, n, stream)
    torch.cuda.synchronize()        # the plain FP32 absmax (q.scales) is freed on return
    return n


# ----------------------------------------------------------------------------
# one wrapper per entry point
# ----------------------------------------------------------------------------
def bqm_abi_version() -> int:
    return load().bqm_abi_version()


def bqm_last_error() -> str:
    return load().bqm_last_error().decode(errors="replace")


def bqm_quantize_nvfp4_workspace_size(n_mat, rows, cols, scale_mode) -> int:
    return load().bqm_quantize_nvfp4_workspace_size(n_mat, rows, cols, scale_mode)


def bqm_quantize_nvfp4(x, four_over_six: int, s_dec_in, out: QTensor, ws=None, stream=None):
    lib = load()
    qc = out.c()
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.bqm_quantize_nvfp4(_ptr(x), int(four_over_six), _ptr(s_dec_in), C.byref(qc), _ptr(ws),
                                  wsb, _stream(stream)))
    out.four_over_six = qc.four_over_six
    return out


def bqm_quantize_nvfp4_noalloc(x, four_over_six: int, s_dec_in, out: QTensor, stream=None):
    lib = load()
    qc = out.c()
    _check(lib.bqm_quantize_nvfp4_noalloc(_ptr(x), int(four_over_six), _ptr(s_dec_in), C.byref(qc),
                                          _stream(stream)))
    out.four_over_six = qc.four_over_six
    return out


def bqm_quantize_nf4(x, out: QTensor, stream=None):
    lib = load()
    qc = out.c()
    _check(lib.bqm_quantize_nf4(_ptr(x), C.byref(qc), _stream(stream)))
    return out


def bqm_nf4_nest(plain: QTensor, nested: QTensor, stream=None):
    lib = load()
    pc, nc = plain.c(), nested.c()
    _check(lib.bqm_nf4_nest(C.byref(pc), C.byref(nc), _stream(stream)))
    return nested


def bqm_dequantize(q: QTensor, y, stream=None):
    if q.fmt == FMT_MXFP4:      # checked as the other MXFP4 calls check theirs
        lib, dev = _begin()
        _check(lib.bqm_dequantize(_mxfp4("q", q, dev), _dense("y", y, _bf16, q.n_mat * q.rows * q.cols, dev),
                                  _stream(stream)))
        return y
    lib = load()
    qc = q.c()
    _check(lib.bqm_dequantize(C.byref(qc), _ptr(y), _stream(stream)))
    return y


def bqm_route(logits, T, E, k, renorm, topk_idx, topk_w, stream=None):
    _check(load().bqm_route(_ptr(logits), T, E, k, int(renorm), _ptr(topk_idx), _ptr(topk_w),
                            _stream(stream)))


def bqm_permute_workspace_size(T, E, k) -> int:
    return load().bqm_permute_workspace_size(T, E, k)


def bqm_permute(topk_idx, T, E, k, perm, inv, offsets, ws, stream=None):
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().bqm_permute(_ptr(topk_idx), T, E, k, _ptr(perm), _ptr(inv), _ptr(offsets),
                              _ptr(ws), wsb, _stream(stream)))


@dataclass
class MoEDesc:
    T: int
    H: int
    I: int
    E: int
    k: int
    r: int
    w_gu: QTensor
    w_dn: QTensor
    A_gu: object = None
    B_gu: object = None
    A_dn: object = None
    B_dn: object = None
    lora_scale: float = 1.0
    act_quant: int = 0
    stage_events: Optional[int] = None   # address of a host array of 2*STAGE_COUNT hipEvent_t
    lora_shared_a: int = 0               # 1: A_gu [r, H] and A_dn [r, I] shared by all experts

    def c(self) -> MoEDescC:
        return MoEDescC(self.T, self.H, self.I, self.E, self.k, self.r, int(self.act_quant),
                        float(self.lora_scale), int(self.lora_shared_a), self.w_gu.c(), self.w_dn.c(), _ptr(self.A_gu),
                        _ptr(self.B_gu), _ptr(self.A_dn), _ptr(self.B_dn), self.stage_events)


def bqm_moe_workspace_size(d: MoEDesc) -> int:
    dc = d.c()
    return load().bqm_moe_workspace_size(C.byref(dc))


def bqm_moe_fwd(d: MoEDesc, x, topk_idx, topk_w, out, ws, stream=None):
    dc = d.c()
    _check(load().bqm_moe_fwd(C.byref(dc), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(out), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)))


def bqm_moe_dgrad(d: MoEDesc, dy, ws, dx, dtopk_w=None, stream=None):
    dc = d.c()
    _check(load().bqm_moe_dgrad(C.byref(dc), _ptr(dy), _ptr(ws), ws.numel() * ws.element_size(),
                                _ptr(dx), _ptr(dtopk_w), _stream(stream)))


def bqm_moe_dgrad_colwise(d: MoEDesc, w_gu_col: QTensor, w_dn_col: QTensor, dy, ws, dx, dtopk_w=None, stream=None):
    dc = d.c()
    gc, nc = w_gu_col.c(), w_dn_col.c()
    _check(load().bqm_moe_dgrad_colwise(C.byref(dc), C.byref(gc), C.byref(nc), _ptr(dy), _ptr(ws),
                                        ws.numel() * ws.element_size(), _ptr(dx), _ptr(dtopk_w), _stream(stream)))


def bqm_lora_grad(d: MoEDesc, x, dy, ws, dA_gu, dB_gu, dA_dn, dB_dn, stream=None):
    dc = d.c()
    _check(load().bqm_lora_grad(C.byref(dc), _ptr(x), _ptr(dy), _ptr(ws), ws.numel() * ws.element_size(),
                                _ptr(dA_gu), _ptr(dB_gu), _ptr(dA_dn), _ptr(dB_dn), _stream(stream)))


# ----------------------------------------------------------------------------
# experts over MXFP4, the router's training, rows between token and expert order, the dense
# product.  These calls take their sizes from the tensors, so the tensors' types, shapes and
# layout are checked here; everything else is checked behind the C ABI.
# ----------------------------------------------------------------------------
_torch = _bf16 = _f32 = _i32 = _u8 = None


def _begin():
    """The library and the current device (where kernels are launched; -2 without a GPU)."""
    global _torch, _bf16, _f32, _i32, _u8
    if _torch is None:
        import torch
        _bf16, _f32, _i32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
        _torch = torch      # last: another thread that finds it finds the others
    lib = load()
    try:
        return lib, _torch._C._cuda_getDevice()
    except AttributeError:          # not part of torch's public interface
        return lib, _torch.cuda.current_device() if _torch.cuda.is_available() else -2
    except RuntimeError:
        return lib, -2


def _dense(name, t, dtype, n, dev):
    """Address of t (None: None) if it is a contiguous tensor of n elements of that dtype on dev.
    The checks of a short call take as long as its kernel runs, so they are one expression."""
    if t is None:
        return None
    if t.dtype is dtype and t.numel() == n and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    name = ".".join(name) if isinstance(name, tuple) else name
    if t.dtype is not dtype:
        raise BQMError(-1, f"{name}: dtype {t.dtype}, {dtype} needed")
    if not t.is_contiguous():
        raise BQMError(-2, f"{name}: not contiguous")
    if t.numel() != n:
        raise BQMError(-2, f"{name}: shape {tuple(t.shape)}, {n} elements needed")
    if t.get_device() < 0:
        raise BQMError(-1, f"{name}: not a GPU tensor")
    raise BQMError(-1, f"{name}: on device {t.get_device()}, the current one is {dev}")


def _mxfp4(name, q: QTensor, dev):
    if q.fmt != FMT_MXFP4:
        raise BQMError(-1, f"{name}: format {q.fmt}, FMT_MXFP4 needed")
    n = q.n_mat * q.rows * q.cols
    return C.byref(QTensorC(FMT_MXFP4, 0, q.n_mat, q.rows, q.cols, _dense((name, "codes"), q.codes, _u8, n // 2, dev),
                            _dense((name, "scales"), q.scales, _u8, n // 32, dev), None, 0, 0))


def bqm_quantize_mxfp4(x, out: QTensor, stream=None):
    """bf16 x [n_mat, rows, cols] -> out, an MXFP4 stack (returned)."""
    lib, dev = _begin()
    _check(lib.bqm_quantize_mxfp4(_dense("x", x, _bf16, out.n_mat * out.rows * out.cols, dev), _mxfp4("out", out, dev),
                                  _stream(stream)))
    return out


def bqm_mxfp4_gemm(x: QTensor, w: QTensor, offsets, perm, k, y, stream=None):
    """y [R, N] = rows of x [1, rows, K] times their experts' w [E, N, K]; perm None: rows
    are in routed order already.  R is y's first dimension."""
    lib, dev = _begin()
    R = y.shape[0]
    _check(lib.bqm_mxfp4_gemm(_mxfp4("x", x, dev), _mxfp4("w", w, dev), _dense("offsets", offsets, _i32, w.n_mat + 1, dev),
                              _dense("perm", perm, _i32, R, dev), k, R, _dense("y", y, _bf16, R * w.rows, dev),
                              _stream(stream)))
    return y


def bqm_mxfp4_dgrad(w: QTensor, dy, offsets, perm, k, dx, stream=None):
    """dx [R, K] = rows of dy [rows, N] times their experts' DQ(w) [E, N, K]."""
    lib, dev = _begin()
    R, rows = dx.shape[0], dy.shape[0]
    _check(lib.bqm_mxfp4_dgrad(_mxfp4("w", w, dev), _dense("dy", dy, _bf16, rows * w.rows, dev), rows,
                               _dense("offsets", offsets, _i32, w.n_mat + 1, dev), _dense("perm", perm, _i32, R, dev), k,
                               R, _dense("dx", dx, _bf16, R * w.cols, dev), _stream(stream)))
    return dx


def bqm_swiglu_ckpt_fwd(h, h8, h8_scales, a=None, aq: Optional[QTensor] = None, n_rows=None, stream=None):
    """h [R, 2I] -> the 8-bit copy h8 [R, 2I], h8_scales [R, 2I/32]; a [R, I], aq [1, R, I]
    where given.  n_rows: a one-element int32 tensor (offsets[E:], say)."""
    lib, dev = _begin()
    R, I2 = h.shape
    I, n = I2 // 2, R * I2
    _check(lib.bqm_swiglu_ckpt_fwd(_dense("h", h, _bf16, R * 2 * I, dev), R, I, _dense("n_rows", n_rows, _i32, 1, dev),
                                   _dense("h8", h8, _u8, n, dev), _dense("h8_scales", h8_scales, _u8, n // 32, dev),
                                   _dense("a", a, _bf16, R * I, dev), None if aq is None else _mxfp4("aq", aq, dev),
                                   _stream(stream)))


def bqm_swiglu_ckpt_bwd(h8, h8_scales, da, perm, topk_w, dh, dtopk_w=None, n_rows=None, stream=None):
    """The 8-bit copy and da [R, I] -> dh [R, 2I], dtopk_w [R] (or [T, k]) where given."""
    lib, dev = _begin()
    R, I = da.shape
    n = R * I
    _check(lib.bqm_swiglu_ckpt_bwd(_dense("h8", h8, _u8, 2 * n, dev), _dense("h8_scales", h8_scales, _u8, 2 * n // 32, dev),
                                   _dense("da", da, _bf16, n, dev), _dense("perm", perm, _i32, R, dev),
                                   _dense("topk_w", topk_w, _f32, R, dev), R, I, _dense("n_rows", n_rows, _i32, 1, dev),
                                   _dense("dh", dh, _bf16, 2 * n, dev), _dense("dtopk_w", dtopk_w, _f32, R, dev),
                                   _stream(stream)))
    return dh


def bqm_router_loss_workspace_size(T, E) -> int:
    return load().bqm_router_loss_workspace_size(T, E)


def bqm_router_loss(logits, topk_idx, valid, counts, loss, ws, stream=None):
    """logits [T, E], topk_idx [T, k] (valid uint8 [T] or None) -> counts int32 [E+1], loss
    float32 [2] = (balance loss, z-loss).  ws: uint8, bqm_router_loss_workspace_size(T, E)."""
    lib, dev = _begin()
    (T, E), k = logits.shape, topk_idx.shape[1]
    wsb = 0 if ws is None else ws.numel()
    _check(lib.bqm_router_loss(_dense("logits", logits, _f32, T * E, dev), _dense("topk_idx", topk_idx, _i32, T * k, dev),
                               _dense("valid", valid, _u8, T, dev), T, E, k, _dense("counts", counts, _i32, E + 1, dev),
                               _dense("loss", loss, _f32, 2, dev), _dense("ws", ws, _u8, wsb, dev), wsb, _stream(stream)))


def bqm_router_grad(logits, topk_idx, valid, counts, dtopk_w, dloss, renorm, dlogits, stream=None):
    """dlogits [T, E] of the losses (times dloss [2], or None) and of topk_w (times dtopk_w
    [T, k], or None)."""
    lib, dev = _begin()
    (T, E), k = logits.shape, topk_idx.shape[1]
    _check(lib.bqm_router_grad(_dense("logits", logits, _f32, T * E, dev), _dense("topk_idx", topk_idx, _i32, T * k, dev),
                               _dense("valid", valid, _u8, T, dev), _dense("counts", counts, _i32, E + 1, dev),
                               _dense("dtopk_w", dtopk_w, _f32, T * k, dev), _dense("dloss", dloss, _f32, 2, dev), T, E, k,
                               int(renorm), _dense("dlogits", dlogits, _f32, T * E, dev), _stream(stream)))
    return dlogits


def _pairs(name, rows, T):
    """Pairs per token of a tensor [T * k, H] (or inv [T, k], flattened or not)."""
    if T and rows and rows % T == 0:
        return rows // T
    if T == 0 and rows == 0:
        return 1
    raise BQMError(-2, f"{name}: {rows} pairs for {T} tokens")


def bqm_dispatch(x, inv, rows, n_rows=None, stream=None):
    """rows [R, H]: x [T, H] at the place inv [T, k] of each pair.  n_rows: a one-element int32
    tensor (offsets[E:], say); pairs whose place lies behind it are dropped."""
    lib, dev = _begin()
    T, H = x.shape
    R = inv.numel()
    k = _pairs("inv", R, T)
    _check(lib.bqm_dispatch(_dense("x", x, _bf16, T * H, dev), _dense("inv", inv, _i32, R, dev), T, H, k,
                            _dense("n_rows", n_rows, _i32, 1, dev), _dense("rows", rows, _bf16, R * H, dev),
                            _stream(stream)))
    return rows


def bqm_combine(y, inv, out, topk_w=None, residual=None, n_rows=None, stream=None):
    """out [T, H]: each token's rows of y [R, H] times topk_w [T, k] (None: 1), plus residual."""
    lib, dev = _begin()
    T, H = out.shape
    R = inv.numel()
    k = _pairs("inv", R, T)
    _check(lib.bqm_combine(_dense("y", y, _bf16, R * H, dev), _dense("inv", inv, _i32, R, dev),
                           _dense("topk_w", topk_w, _f32, R, dev), _dense("residual", residual, _bf16, T * H, dev), T, H,
                           k, _dense("n_rows", n_rows, _i32, 1, dev), _dense("out", out, _bf16, T * H, dev),
                           _stream(stream)))
    return out


def bqm_combine_grad(dout, inv, y=None, topk_w=None, dy=None, dtopk_w=None, n_rows=None, stream=None):
    """dout [T, H] -> dy [R, H] and dtopk_w [T, k] (which needs y [R, H]), where given; dy may be
    y where no two pairs stand at one row."""
    lib, dev = _begin()
    T, H = dout.shape
    R = inv.numel()
    k = _pairs("inv", R, T)
    _check(lib.bqm_combine_grad(_dense("dout", dout, _bf16, T * H, dev), _dense("y", y, _bf16, R * H, dev),
                                _dense("inv", inv, _i32, R, dev), _dense("topk_w", topk_w, _f32, R, dev), T, H, k,
                                _dense("n_rows", n_rows, _i32, 1, dev), _dense("dy", dy, _bf16, R * H, dev),
                                _dense("dtopk_w", dtopk_w, _f32, R, dev), _stream(stream)))


def bqm_linear_workspace_size(M, N, K) -> int:
    """Bytes of ws for the three products with weights [N, K] and up to M rows."""
    return load().bqm_linear_workspace_size(M, N, K)


def bqm_linear_fwd(x, w, y, bias=None, act=ACT_NONE, residual=None, z=None, ws=None, stream=None):
    """y [M, N] = act(x [M, K] w [N, K]^T + bias [N]) + residual [M, N]; z [M, N]: the
    pre-activation, where given.  ws: uint8, bqm_linear_workspace_size(M, N, K)."""
    lib, dev = _begin()
    (M, K), N = x.shape, w.shape[0]
    wsb = 0 if ws is None else ws.numel()
    _check(lib.bqm_linear_fwd(_dense("x", x, _bf16, M * K, dev), _dense("w", w, _bf16, N * K, dev),
                              _dense("bias", bias, _bf16, N, dev), act, _dense("residual", residual, _bf16, M * N, dev), M,
                              N, K, _dense("y", y, _bf16, M * N, dev), _dense("z", z, _bf16, M * N, dev),
                              _dense("ws", ws, _u8, wsb, dev), wsb, _stream(stream)))
    return y


def bqm_linear_dgrad(dz, w, dx, zx=None, act=ACT_NONE, add=None, ws=None, stream=None):
    """dx [M, K] = dz [M, N] w [N, K], times act'(zx [M, K]) with an activation, plus add [M, K]."""
    lib, dev = _begin()
    (N, K), M = w.shape, dz.shape[0]
    wsb = 0 if ws is None else ws.numel()
    _check(lib.bqm_linear_dgrad(_dense("dz", dz, _bf16, M * N, dev), _dense("w", w, _bf16, N * K, dev),
                                _dense("zx", zx, _bf16, M * K, dev), act, _dense("add", add, _bf16, M * K, dev), M, N, K,
                                _dense("dx", dx, _bf16, M * K, dev), _dense("ws", ws, _u8, wsb, dev), wsb,
                                _stream(stream)))
    return dx


def bqm_linear_wgrad(dz, x, dw, dbias=None, accumulate=False, ws=None, stream=None):
    """dw float32 [N, K] = dz [M, N]^T x [M, K], dbias float32 [N] = the sum of dz's rows; added
    to what they hold with accumulate."""
    lib, dev = _begin()
    (M, N), K = dz.shape, x.shape[1]
    wsb = 0 if ws is None else ws.numel()
    _check(lib.bqm_linear_wgrad(_dense("dz", dz, _bf16, M * N, dev), _dense("x", x, _bf16, M * K, dev), int(accumulate), M,
                                N, K, _dense("dw", dw, _f32, N * K, dev), _dense("dbias", dbias, _f32, N, dev),
                                _dense("ws", ws, _u8, wsb, dev), wsb, _stream(stream)))
    return dw


def bqm_act_grad(dy, z, act, dz, stream=None):
    """dz = dy act'(z), element by element."""
    lib, dev = _begin()
    n = dy.numel()
    _check(lib.bqm_act_grad(_dense("dy", dy, _bf16, n, dev), _dense("z", z, _bf16, n, dev), act, n,
                            _dense("dz", dz, _bf16, n, dev), _stream(stream)))
    return dz
