"""Python binding of libiq (block-scaled quantization on MI355X).

A thin ctypes layer over the C ABI declared in include/iq.h: the functions
below carry the C names and only marshal arguments (_fast.so does the same for
short calls).  torch provides device
memory (torch.empty) and the current HIP stream; every step of quantization
runs in the HIP kernels of libiq.so.  There is no CPU fallback: importing
works anywhere, but any call raises if the library is missing.

With `stream` a call runs on that stream, and what it allocates (results and
workspace) belongs to it, as under `with torch.cuda.stream(stream)`.

The feed-forward operators record no graph: gradients come from the *_backward
functions, and tensors that require gradients are refused outside no_grad().
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libiq.so")

# iq_format / iq_gran / iq_dtype / iq_status values of include/iq.h
FORMATS = {"int8": 0, "e4m3": 1, "e5m2": 2, "mxfp4": 3, "nvfp4": 4, "int4": 5, "int4zp": 6}
GRANS = {"tensor": 0, "row": 1, "block": 2}
IQ_F32, IQ_BF16 = 0, 1
IQ_OK, IQ_EINVAL, IQ_EALIGN, IQ_EUNSUPPORTED, IQ_EHIP = 0, 1, 2, 3, 4
# iq_desc.flags: scale-rule variants (MXFP4 exponent rounding, NVFP4 block-scale rounding)
IQ_FLAG_MX_ROUND_NEAREST, IQ_FLAG_MX_ROUND_UP, IQ_FLAG_NV_SCALE_RNE = 0x1, 0x2, 0x4
# iq_act values
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
FOUR_BIT = ("mxfp4", "nvfp4", "int4", "int4zp")


class IQDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("gran", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("reserved0", ctypes.c_int32), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld_in", ctypes.c_int64), ("flags", ctypes.c_uint32), ("reserved1", ctypes.c_uint32)]


class IQGatedDesc(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("dtype", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("features", ctypes.c_int64), ("ld_x", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class IQStats(ctypes.Structure):
    _fields_ = [("n", ctypes.c_uint64), ("n_zero_flush", ctypes.c_uint64),
                ("n_saturated", ctypes.c_uint64), ("n_nonfinite", ctypes.c_uint64),
                ("sum_x2", ctypes.c_double), ("sum_err2", ctypes.c_double),
                ("sum_abs_err", ctypes.c_double), ("max_abs_err", ctypes.c_float),
                ("reserved", ctypes.c_uint32)]

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_ if k != "reserved"}


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libiq.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"libiq.so not found at {path}: build it with __graft_entry__.build()")
    L = ctypes.CDLL(path)
    P, S = ctypes.c_void_p, ctypes.c_size_t
    D = ctypes.POINTER(IQDesc)
    L.iq_codes_bytes.restype, L.iq_codes_bytes.argtypes = S, [D]
    L.iq_scales_bytes.restype, L.iq_scales_bytes.argtypes = S, [D]
    L.iq_workspace_bytes.restype, L.iq_workspace_bytes.argtypes = S, [D]
    L.iq_quantize.restype = ctypes.c_int
    L.iq_quantize.argtypes = [D, P, P, P, P, P, P, ctypes.c_int32, P, P]
    L.iq_quantize_noalloc.restype = ctypes.c_int
    L.iq_quantize_noalloc.argtypes = [D, P, P, P, P, P, P, ctypes.c_int32, P]
    L.iq_quantize_static.restype = ctypes.c_int
    L.iq_quantize_static.argtypes = [D, P, P, P, P, P, P, P, ctypes.c_int32, P, P]
    L.iq_quantize_zp.restype = ctypes.c_int
    L.iq_quantize_zp.argtypes = [D, P, P, P, P, P, P, ctypes.c_int32, P, P]
    L.iq_dequantize_zp.restype = ctypes.c_int
    L.iq_dequantize_zp.argtypes = [D, P, P, P, P, ctypes.c_int32, P]
    L.iq_shifts_bytes.restype, L.iq_shifts_bytes.argtypes = S, [D]
    L.iq_zp_gemm.restype = ctypes.c_int
    L.iq_zp_gemm.argtypes = [D, P, P, P, P, ctypes.c_int32, ctypes.c_int64, P, P]
    L.iq_mx_gemm.restype = ctypes.c_int
    L.iq_mx_gemm.argtypes = [D, P, P, P, P, ctypes.c_int64, P, P]
    L.iq_mxw_gemm.restype = ctypes.c_int
    L.iq_mxw_gemm.argtypes = [D, P, P, P, ctypes.c_int32, ctypes.c_int64, P, P]
    L.iq_dequantize.restype = ctypes.c_int
    L.iq_dequantize.argtypes = [D, P, P, P, P, ctypes.c_int32, P]
    L.iq_amax.restype = ctypes.c_int
    L.iq_amax.argtypes = [D, P, P, P, P]
    I, N, F = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    G = ctypes.POINTER(IQGatedDesc)
    L.iq_layer_norm.restype = ctypes.c_int
    L.iq_layer_norm.argtypes = [D, P, P, P, I, F, P, P, P, P]
    L.iq_layer_norm_backward.restype = ctypes.c_int
    L.iq_layer_norm_backward.argtypes = [D, P, P, P, I, P, P, P, P, P, P, P]
    L.iq_layer_norm_workspace_bytes.restype, L.iq_layer_norm_workspace_bytes.argtypes = S, [D]
    L.iq_gated_forward.restype = ctypes.c_int
    L.iq_gated_forward.argtypes = [G, P, P, P, P, P, P]
    L.iq_gated_backward.restype = ctypes.c_int
    L.iq_gated_backward.argtypes = [G, P, P, P, P, P, P, P, P, P, P]
    L.iq_gated_saved_bytes.restype, L.iq_gated_saved_bytes.argtypes = S, [G]
    L.iq_gated_workspace_bytes.restype, L.iq_gated_workspace_bytes.argtypes = S, [G]
    L.iq_packed_gemv.restype = ctypes.c_int
    L.iq_packed_gemv.argtypes = [D, P, P, P, P, I, N, P, I, P]
    L.iq_packed_gated.restype = ctypes.c_int
    L.iq_packed_gated.argtypes = [D, I, P, P, P, P, P, P, P, I, N, P, I, P]
    L.iq_status_str.restype, L.iq_status_str.argtypes = ctypes.c_char_p, [ctypes.c_int]
    L.iq_abi_version.restype, L.iq_abi_version.argtypes = ctypes.c_int, []
    _lib = L
    return L


class IQError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {iq_status_str(status)} ({status})")
        self.status = status


def _check(status: int, what: str) -> None:
    if status != IQ_OK:
        raise IQError(status, what)


# ---- C entry points (same names, marshalling only) -------------------------
def iq_abi_version() -> int:
    return load_library().iq_abi_version()


def iq_status_str(status: int) -> str:
    return load_library().iq_status_str(status).decode()


def iq_codes_bytes(d: IQDesc) -> int:
    return load_library().iq_codes_bytes(ctypes.byref(d))


def iq_scales_bytes(d: IQDesc) -> int:
    return load_library().iq_scales_bytes(ctypes.byref(d))


def iq_workspace_bytes(d: IQDesc) -> int:
    return load_library().iq_workspace_bytes(ctypes.byref(d))


def iq_quantize(d: IQDesc, x: int, codes: int, scales: int, global_scale: int | None, stats: int | None,
                xhat: int | None, xhat_dtype: int, workspace: int, stream: int | None) -> int:
    """Raw call with integer device addresses; returns the iq_status."""
    return load_library().iq_quantize(ctypes.byref(d), x, codes, scales, global_scale, stats, xhat,
                                      xhat_dtype, workspace, stream)


def iq_quantize_noalloc(d: IQDesc, x: int, codes: int, scales: int, global_scale: int | None, stats: int | None,
                        xhat: int | None, xhat_dtype: int, stream: int | None) -> int:
    """Raw call with integer device addresses; the library's own workspace."""
    return load_library().iq_quantize_noalloc(ctypes.byref(d), x, codes, scales, global_scale, stats, xhat,
                                              xhat_dtype, stream)


def iq_quantize_static(d: IQDesc, x: int, amax_in: int, codes: int, scales: int, global_scale: int | None,
                       stats: int | None, xhat: int | None, xhat_dtype: int, workspace: int,
                       stream: int | None) -> int:
    """Raw call with integer device addresses (amax_in: device float32 [1])."""
    return load_library().iq_quantize_static(ctypes.byref(d), x, amax_in, codes, scales, global_scale, stats,
                                             xhat, xhat_dtype, workspace, stream)


def iq_quantize_zp(d: IQDesc, x: int, codes: int, scales: int, shifts: int, stats: int | None,
                   xhat: int | None, xhat_dtype: int, workspace: int, stream: int | None) -> int:
    return load_library().iq_quantize_zp(ctypes.byref(d), x, codes, scales, shifts, stats, xhat, xhat_dtype,
                                         workspace, stream)


def iq_dequantize_zp(d: IQDesc, codes: int, scales: int, shifts: int, xhat: int, xhat_dtype: int,
                     stream: int | None) -> int:
    return load_library().iq_dequantize_zp(ctypes.byref(d), codes, scales, shifts, xhat, xhat_dtype, stream)


def iq_shifts_bytes(d: IQDesc) -> int:
    return load_library().iq_shifts_bytes(ctypes.byref(d))


def iq_zp_gemm(d: IQDesc, codes: int, scales: int, shifts: int, x: int, x_dtype: int, n1: int, z: int,
               stream: int | None) -> int:
    return load_library().iq_zp_gemm(ctypes.byref(d), codes, scales, shifts, x, x_dtype, n1, z, stream)


def iq_mx_gemm(d: IQDesc, codes_w: int, scales_w: int, codes_a: int, scales_a: int, n1: int, z: int,
               stream: int | None) -> int:
    return load_library().iq_mx_gemm(ctypes.byref(d), codes_w, scales_w, codes_a, scales_a, n1, z, stream)


def iq_mxw_gemm(d: IQDesc, codes: int, scales: int, x: int, x_dtype: int, n1: int, z: int,
                stream: int | None) -> int:
    return load_library().iq_mxw_gemm(ctypes.byref(d), codes, scales, x, x_dtype, n1, z, stream)


def iq_dequantize(d: IQDesc, codes: int, scales: int, global_scale: int | None, xhat: int,
                  xhat_dtype: int, stream: int | None) -> int:
    return load_library().iq_dequantize(ctypes.byref(d), codes, scales, global_scale, xhat, xhat_dtype,
                                        stream)


def iq_amax(d: IQDesc, x: int, amax_out: int, workspace: int, stream: int | None) -> int:
    return load_library().iq_amax(ctypes.byref(d), x, amax_out, workspace, stream)


def iq_layer_norm(d: IQDesc, x: int, weight: int | None, bias: int | None, param_dtype: int, eps: float, y: int,
                  mean: int | None, rstd: int | None, stream: int | None) -> int:
    return (_lib or load_library()).iq_layer_norm(ctypes.byref(d), x, weight, bias, param_dtype, eps, y, mean, rstd, stream)


def iq_layer_norm_backward(d: IQDesc, x: int, dy: int, weight: int | None, param_dtype: int, mean: int, rstd: int,
                           dx: int | None, dweight: int | None, dbias: int | None, workspace: int | None,
                           stream: int | None) -> int:
    return (_lib or load_library()).iq_layer_norm_backward(ctypes.byref(d), x, dy, weight, param_dtype, mean, rstd, dx,
                                                 dweight, dbias, workspace, stream)


def iq_layer_norm_workspace_bytes(d: IQDesc) -> int:
    return (_lib or load_library()).iq_layer_norm_workspace_bytes(ctypes.byref(d))


def iq_gated_forward(d: IQGatedDesc, x: int, w_gate: int, w_up: int, h: int, saved: int | None,
                     stream: int | None) -> int:
    return (_lib or load_library()).iq_gated_forward(ctypes.byref(d), x, w_gate, w_up, h, saved, stream)


def iq_gated_backward(d: IQGatedDesc, dh: int, x: int, w_gate: int, w_up: int, saved: int, dx: int | None,
                      dw_gate: int | None, dw_up: int | None, workspace: int, stream: int | None) -> int:
    return (_lib or load_library()).iq_gated_backward(ctypes.byref(d), dh, x, w_gate, w_up, saved, dx, dw_gate, dw_up,
                                            workspace, stream)


def iq_gated_saved_bytes(d: IQGatedDesc) -> int:
    return load_library().iq_gated_saved_bytes(ctypes.byref(d))


def iq_gated_workspace_bytes(d: IQGatedDesc) -> int:
    return (_lib or load_library()).iq_gated_workspace_bytes(ctypes.byref(d))


def iq_packed_gemv(d: IQDesc, codes: int, scales: int, global_scale: int | None, x: int, x_dtype: int, n1: int,
                   z: int, z_dtype: int, stream: int | None) -> int:
    return (_lib or load_library()).iq_packed_gemv(ctypes.byref(d), codes, scales, global_scale, x, x_dtype, n1, z, z_dtype,
                                         stream)


def iq_packed_gated(d: IQDesc, act: int, codes_gate: int, scales_gate: int, global_gate: int | None, codes_up: int,
                    scales_up: int, global_up: int | None, x: int, x_dtype: int, n1: int, h: int, h_dtype: int,
                    stream: int | None) -> int:
    return (_lib or load_library()).iq_packed_gated(ctypes.byref(d), act, codes_gate, scales_gate, global_gate, codes_up,
                                          scales_up, global_up, x, x_dtype, n1, h, h_dtype, stream)


# ---- torch-facing helpers (allocation with torch.empty + the calls above) ---
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def make_desc(fmt: str, gran: str, rows: int, cols: int, in_dtype: int = IQ_BF16, ld: int | None = None,
              flags: int = 0) -> IQDesc:
    return IQDesc(FORMATS[fmt], GRANS[gran], in_dtype, 0, rows, cols, cols if ld is None else ld, flags, 0)


def desc_for(x, fmt: str, gran: str, cols: int | None = None, flags: int = 0) -> IQDesc:
    """Descriptor of a 2-D CUDA/HIP tensor (float32 or bfloat16, unit column stride)."""
    torch = _torch()
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype == torch.float32:
        dt = IQ_F32
    elif x.dtype == torch.bfloat16:
        dt = IQ_BF16
    else:
        raise TypeError("x must be float32 or bfloat16")
    rows = x.shape[0]
    c = x.shape[1] if cols is None else cols
    ld = x.stride(0) if rows > 1 else c   # a single row is read at ld-independent offsets
    return IQDesc(FORMATS[fmt], GRANS[gran], dt, 0, rows, c, ld, flags, 0)


_here = contextlib.nullcontext()


def _place(stream, x):
    """What a call on x allocates and launches inside belongs to `stream`, or
    to the current stream of x's device where none is named.  Memory of another
    stream could be taken back, or still be in use there, while the call runs."""
    torch = _torch()
    if stream is None:
        if not x.is_cuda or x.get_device() == torch._C._cuda_getDevice():
            return _here
        return torch.cuda.device(x.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, x.device)
    if stream.device != x.device:
        raise ValueError(f"x is on {x.device}, the stream on {stream.device}")
    return torch.cuda.stream(stream)


def _stream_for(x):
    """The stream that a call on x runs on, inside `_place`; x has to be in GPU memory."""
    if not x.is_cuda:
        raise ValueError(f"x is on {x.device}, not on a GPU")
    return _torch()._C._cuda_getCurrentRawStream(x.get_device())     # current_stream() without its object


def _ptr(t):
    return None if t is None else t.data_ptr()


def empty_outputs(d: IQDesc, device, fmt: str, gran: str):
    """codes, scales, global_scale tensors for a descriptor (torch.empty)."""
    torch = _torch()
    rows, cols = d.rows, d.cols
    codes = torch.empty((rows, cols // 2 if fmt in FOUR_BIT else cols), dtype=torch.uint8, device=device)
    if fmt in ("int8", "e4m3", "e5m2"):
        scales = torch.empty((1,) if gran == "tensor" else (rows,), dtype=torch.float32, device=device)
    elif fmt == "mxfp4":
        scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=device)
    elif fmt == "nvfp4":
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=device)
    elif fmt == "int4zp":
        scales = torch.empty((rows, cols // 128), dtype=torch.float32, device=device)
    else:
        scales = torch.empty((rows, cols // 128), dtype=torch.int16, device=device)
    gscale = torch.empty((1,), dtype=torch.float32, device=device) if fmt == "nvfp4" else None
    return codes, scales, gscale


def workspace_for(d: IQDesc, device):
    """A zero-filled workspace (the library's tickets start at zero and every
    call leaves them there); 256-byte aligned."""
    torch = _torch()
    n = iq_workspace_bytes(d)
    return torch.zeros((n + 255) // 256 * 64, dtype=torch.float32, device=device)


def _check_buffer(t, nbytes: int, what: str, device, dtype=None):
    """A caller-supplied device buffer must be contiguous, on the input's
    device, of the expected dtype and hold at least nbytes."""
    if t is None:
        raise ValueError(f"{what} is missing")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the input on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{what} holds {t.numel() * t.element_size()} bytes, needs {nbytes}")


def _check_out(out: "Quantized", d: IQDesc, fmt: str, gran: str, device):
    """A Quantized passed as `out` must match the descriptor of this call."""
    torch = _torch()
    if out.fmt != fmt or out.gran != gran or out.rows != d.rows or out.cols != d.cols:
        raise ValueError("out was made for another format, granularity or shape")
    _check_buffer(out.codes, iq_codes_bytes(d), "out.codes", device, torch.uint8)
    _check_buffer(out.scales, iq_scales_bytes(d), "out.scales", device)
    if fmt == "nvfp4":
        _check_buffer(out.global_scale, 4, "out.global_scale", device, torch.float32)
    if fmt == "int4zp":
        _check_buffer(out.shifts, iq_shifts_bytes(d), "out.shifts", device, torch.uint8)
    if out.stats_buf is not None:
        _check_buffer(out.stats_buf, ctypes.sizeof(IQStats), "out.stats_buf", device)
    if out.xhat is not None:
        if out.xhat.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("out.xhat must be float32 or bfloat16")
        _check_buffer(out.xhat, d.rows * d.cols * out.xhat.element_size(), "out.xhat", device)


@dataclass
class Quantized:
    codes: object
    scales: object
    global_scale: object
    xhat: object
    stats_buf: object
    fmt: str
    gran: str
    rows: int
    cols: int
    shifts: object = None   # asymmetric INT4: uint8 [rows, cols / 256]

    def stats(self) -> dict:
        """Copy the statistics to the host (synchronizes with the device)."""
        if self.stats_buf is None:
            return None
        raw = bytes(self.stats_buf.cpu().numpy().tobytes())
        return IQStats.from_buffer_copy(raw).as_dict()


def quantize(x, fmt: str, gran: str, *, stats: bool = True, xhat_dtype=None, cols: int | None = None,
             flags: int = 0, workspace=None, out=None, stream=None, static_amax=None) -> Quantized:
    """Quantize a device tensor; outputs are allocated with torch.empty unless
    `out` (a Quantized from a previous call of the same shape) is given.
    static_amax (a device float32 tensor of one element) selects static
    scaling: iq_quantize_static with that absmax instead of the measured one."""
    with _place(stream, x):
        torch = _torch()
        d = desc_for(x, fmt, gran, cols, flags)
        if out is None:
            codes, scales, gscale = empty_outputs(d, x.device, fmt, gran)
            sbuf = torch.empty((64,), dtype=torch.uint8, device=x.device) if stats else None
            xh = None
            if xhat_dtype is not None:
                xh = torch.empty((d.rows, d.cols), dtype=xhat_dtype, device=x.device)
            shifts = (torch.empty((d.rows, d.cols // 256), dtype=torch.uint8, device=x.device)
                      if fmt == "int4zp" else None)
            out = Quantized(codes, scales, gscale, xh, sbuf, fmt, gran, d.rows, d.cols, shifts)
        else:
            _check_out(out, d, fmt, gran, x.device)
        if workspace is None:
            ws = workspace_for(d, x.device)
        else:
            _check_buffer(workspace, iq_workspace_bytes(d), "workspace", x.device)
            ws = workspace
        xdt = IQ_F32
        if out.xhat is not None:
            xdt = IQ_F32 if out.xhat.dtype == torch.float32 else IQ_BF16
        if fmt == "int4zp":
            if static_amax is not None:
                raise ValueError("static_amax needs a per-tensor format or NVFP4")
            st = iq_quantize_zp(d, x.data_ptr(), _ptr(out.codes), _ptr(out.scales), _ptr(out.shifts),
                                _ptr(out.stats_buf), _ptr(out.xhat), xdt, ws.data_ptr(), _stream_for(x))
            _check(st, "iq_quantize_zp")
        elif static_amax is None:
            st = iq_quantize(d, x.data_ptr(), _ptr(out.codes), _ptr(out.scales), _ptr(out.global_scale),
                             _ptr(out.stats_buf), _ptr(out.xhat), xdt, ws.data_ptr(), _stream_for(x))
            _check(st, "iq_quantize")
        else:
            if static_amax.dtype != torch.float32 or static_amax.numel() != 1 or static_amax.device != x.device:
                raise ValueError("static_amax must be one float32 on the input's device")
            st = iq_quantize_static(d, x.data_ptr(), static_amax.data_ptr(), _ptr(out.codes), _ptr(out.scales),
                                    _ptr(out.global_scale), _ptr(out.stats_buf), _ptr(out.xhat), xdt,
                                    ws.data_ptr(), _stream_for(x))
            _check(st, "iq_quantize_static")
        return out


def dequantize(q: Quantized, out_dtype=None, out=None, stream=None):
    with _place(stream, q.codes):
        torch = _torch()
        out_dtype = torch.float32 if out_dtype is None else out_dtype
        d = make_desc(q.fmt, q.gran, q.rows, q.cols)
        if out is None:
            out = torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.codes.device)
        elif out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (q.rows, q.cols):
            raise ValueError("out must be a float32 or bfloat16 [rows, cols] tensor")
        else:
            _check_buffer(out, q.rows * q.cols * out.element_size(), "out", q.codes.device)
        _check_buffer(q.codes, iq_codes_bytes(d), "codes", q.codes.device, torch.uint8)
        _check_buffer(q.scales, iq_scales_bytes(d), "scales", q.codes.device)
        if q.fmt == "nvfp4":
            _check_buffer(q.global_scale, 4, "global_scale", q.codes.device, torch.float32)
        if q.fmt == "int4zp":
            _check_buffer(q.shifts, iq_shifts_bytes(d), "shifts", q.codes.device, torch.uint8)
        dt = IQ_F32 if out.dtype == torch.float32 else IQ_BF16
        if q.fmt == "int4zp":
            st = iq_dequantize_zp(d, q.codes.data_ptr(), q.scales.data_ptr(), _ptr(q.shifts), out.data_ptr(), dt,
                                  _stream_for(q.codes))
            _check(st, "iq_dequantize_zp")
            return out
        st = iq_dequantize(d, q.codes.data_ptr(), q.scales.data_ptr(), _ptr(q.global_scale), out.data_ptr(), dt,
                           _stream_for(q.codes))
        _check(st, "iq_dequantize")
        return out


def amax(x, workspace=None, stream=None):
    with _place(stream, x):
        torch = _torch()
        d = desc_for(x, "e4m3", "tensor")
        out = torch.empty((1,), dtype=torch.float32, device=x.device)
        if workspace is None:
            ws = workspace_for(d, x.device)
        else:
            _check_buffer(workspace, iq_workspace_bytes(d), "workspace", x.device)
            ws = workspace
        _check(iq_amax(d, x.data_ptr(), out.data_ptr(), ws.data_ptr(), _stream_for(x)), "iq_amax")
        return out


def _gemm_out(out, n0: int, n1: int, device):
    """z float32 [n0, n1]: a new tensor, or the caller's after checks."""
    torch = _torch()
    if out is None:
        return torch.empty((n0, n1), dtype=torch.float32, device=device)
    if tuple(out.shape) != (n0, n1):
        raise ValueError(f"out must be [{n0}, {n1}], got {tuple(out.shape)}")
    _check_buffer(out, n0 * n1 * 4, "out", device, torch.float32)
    return out


def zp_gemm(q: "Quantized", x, out=None, stream=None):
    """Puzzle 12's z[j, k] = sum_l sc (w - sh) y[l, k] for asymmetric INT4
    weights q (from quantize(..., "int4zp", "block")) and token-major BF16
    activations x [n1, K]; returns z float32 [N0, n1]."""
    with _place(stream, x):
        torch = _torch()
        if q.fmt != "int4zp":
            raise ValueError("zp_gemm needs asymmetric INT4 weights")
        if x.dim() != 2 or x.shape[1] != q.cols or x.dtype != torch.bfloat16 or not x.is_contiguous():
            raise ValueError("x must be a contiguous BF16 [n1, K] tensor")
        n1 = x.shape[0]
        out = _gemm_out(out, q.rows, n1, x.device)
        d = make_desc("int4zp", "block", q.rows, q.cols)
        _check_buffer(q.codes, iq_codes_bytes(d), "codes", x.device, torch.uint8)
        _check_buffer(q.scales, iq_scales_bytes(d), "scales", x.device, torch.float32)
        _check_buffer(q.shifts, iq_shifts_bytes(d), "shifts", x.device, torch.uint8)
        st = iq_zp_gemm(d, q.codes.data_ptr(), q.scales.data_ptr(), q.shifts.data_ptr(), x.data_ptr(), IQ_BF16, n1,
                        out.data_ptr(), _stream_for(x))
        _check(st, "iq_zp_gemm")
        return out


def mx_gemm(qw: "Quantized", qa: "Quantized", out=None, stream=None):
    """FP4 GEMM z[j, t] = sum_k xw[j, k] xa[t, k] of two MXFP4 operands (from
    quantize(..., "mxfp4", "block")), weights qw [N0, K] and activations
    qa [n1, K]; returns z float32 [N0, n1]."""
    with _place(stream, qw.codes):
        torch = _torch()
        if qw.fmt != "mxfp4" or qa.fmt != "mxfp4":
            raise ValueError("mx_gemm needs two MXFP4 operands")
        if qa.cols != qw.cols:
            raise ValueError("operands disagree on K")
        n1 = qa.rows
        out = _gemm_out(out, qw.rows, n1, qw.codes.device)
        d = make_desc("mxfp4", "block", qw.rows, qw.cols)
        da = make_desc("mxfp4", "block", qa.rows, qa.cols)
        dev = qw.codes.device
        _check_buffer(qw.codes, iq_codes_bytes(d), "weight codes", dev, torch.uint8)
        _check_buffer(qw.scales, iq_scales_bytes(d), "weight scales", dev, torch.uint8)
        _check_buffer(qa.codes, iq_codes_bytes(da), "activation codes", dev, torch.uint8)
        _check_buffer(qa.scales, iq_scales_bytes(da), "activation scales", dev, torch.uint8)
        st = iq_mx_gemm(d, qw.codes.data_ptr(), qw.scales.data_ptr(), qa.codes.data_ptr(), qa.scales.data_ptr(), n1,
                        out.data_ptr(), _stream_for(qw.codes))
        _check(st, "iq_mx_gemm")
        return out


def mxw_gemm(qw: "Quantized", x, out=None, stream=None):
    """MXFP4 weights qw [N0, K] (from quantize(..., "mxfp4", "block")) against
    token-major BF16 activations x [n1, K]: z[j, t] = sum_k xw[j, k] x[t, k];
    returns z float32 [N0, n1]."""
    with _place(stream, x):
        torch = _torch()
        if qw.fmt != "mxfp4":
            raise ValueError("mxw_gemm needs MXFP4 weights")
        if x.dim() != 2 or x.shape[1] != qw.cols or x.dtype != torch.bfloat16 or not x.is_contiguous():
            raise ValueError("x must be a contiguous BF16 [n1, K] tensor")
        n1 = x.shape[0]
        out = _gemm_out(out, qw.rows, n1, x.device)
        d = make_desc("mxfp4", "block", qw.rows, qw.cols)
        _check_buffer(qw.codes, iq_codes_bytes(d), "weight codes", x.device, torch.uint8)
        _check_buffer(qw.scales, iq_scales_bytes(d), "weight scales", x.device, torch.uint8)
        st = iq_mxw_gemm(d, qw.codes.data_ptr(), qw.scales.data_ptr(), x.data_ptr(), IQ_BF16, n1, out.data_ptr(),
                         _stream_for(x))
        _check(st, "iq_mxw_gemm")
        return out


# ---- the feed-forward half of a layer ---------------------------------------
# Calls of a few microseconds of GPU time.  The common case (dense tensors on
# the current device, results allocated here, torch's current stream) is
# checked, allocated and called in _fast.so, which returns None for any other;
# the code below it here serves those and says what is wrong.
_fast_calls = None


def _bind_fast():
    """The module of _fast.so, bound to the loaded library."""
    global _fast_calls
    if _fast_calls is None:
        import importlib
        lib = load_library()
        _torch()
        path = os.path.join(_HERE, "_fast.so")
        if not os.path.exists(path):
            raise OSError(f"_fast.so not found at {path}: build it with __graft_entry__.build()")
        module = importlib.import_module(__name__ + "._fast")
        module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "iq_layer_norm", "iq_layer_norm_backward", "iq_layer_norm_workspace_bytes", "iq_gated_forward",
            "iq_gated_backward", "iq_gated_workspace_bytes", "iq_packed_gemv", "iq_packed_gated")))
        _fast_calls = module
    return _fast_calls


_DTYPES = {}


def _dtypes() -> dict:
    """torch dtype -> iq_dtype."""
    if not _DTYPES:
        torch = _torch()
        _DTYPES.update({torch.float32: IQ_F32, torch.bfloat16: IQ_BF16})
    return _DTYPES


def _dtype_of(t, what: str) -> int:
    code = _dtypes().get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32 or bfloat16")
    return code


def _refuse_grad(*tensors):
    """No graph is recorded, so a tensor that asks for a gradient would never get it."""
    if _torch().is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise RuntimeError("no gradient passes through this call: use tensors without requires_grad or torch.no_grad(), "
                           "and layer_norm_backward or gated_backward for the gradients")


def _result(out, shape: tuple, dtype, x, what: str = "out"):
    """A new tensor on x's device, or the caller's after checks."""
    if out is None:
        return x.new_empty(shape, dtype=dtype)
    _check_dense(out, shape, dtype, x, what)
    return out


def _check_dense(t, shape: tuple, dtype, x, what: str):
    """t is contiguous, of this shape and type and on x's device."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == x.get_device() and t.is_contiguous():
        return
    if tuple(t.shape) != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.device != x.device:
        raise ValueError(f"{what} is on {t.device}, the input on {x.device}")
    raise ValueError(f"{what} must be contiguous")


def _scratch(workspace, nbytes: int, x):
    if workspace is None:
        return x.new_empty((max(nbytes, 256),), dtype=_torch().uint8)
    _check_buffer(workspace, nbytes, "workspace", x.device)
    return workspace


def _norm_desc(x):
    """Descriptor of a layer norm's input (2-D, unit column stride)."""
    if x.dim() != 2 or not (x.is_contiguous() or x.shape[1] == 1 or x.stride(1) == 1):
        raise ValueError("x must be 2-D with unit column stride")
    rows, cols = x.shape
    return IQDesc(0, 0, _dtype_of(x, "x"), 0, rows, cols, x.stride(0) if rows > 1 else cols, 0, 0)


def _norm_params(x, cols: int, weight, bias) -> int:
    """Checks of weight and bias (each [cols] or None); their iq_dtype."""
    first = weight if weight is not None else bias
    if first is None:
        return IQ_F32
    if weight is not None:
        _check_dense(weight, (cols,), first.dtype, x, "weight and bias")
    if bias is not None:
        _check_dense(bias, (cols,), first.dtype, x, "weight and bias")
    return _dtype_of(first, "weight and bias")


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """y = (x - mean) * rstd * weight + bias over the rows of x [rows, cols]
    (float32 or bfloat16, unit column stride); returns y, mean and rstd."""
    if out is None and stream is None:
        done = (_fast_calls or _bind_fast()).layer_norm(x, weight, bias, eps)
        if done is not None:
            return done
    with _place(stream, x):
        _refuse_grad(x, weight, bias, out)
        d = _norm_desc(x)
        rows, cols = d.rows, d.cols
        pt = _norm_params(x, cols, weight, bias)
        y = _torch().empty_like(x) if out is None and x.is_contiguous() else _result(out, (rows, cols), x.dtype, x)
        mean, rstd = x.new_empty((2, rows), dtype=_torch().float32).unbind(0)
        st = iq_layer_norm(d, x.data_ptr(), _ptr(weight), _ptr(bias), pt, eps, y.data_ptr(), mean.data_ptr(),
                           rstd.data_ptr(), _stream_for(x))
        if st:
            _check(st, "iq_layer_norm")
        return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, *, param_dtype=None, workspace=None, stream=None):
    """Gradients of layer_norm: dx of x's type, dweight and dbias of weight's
    (of param_dtype, float32 by default, where weight is None)."""
    if param_dtype is None and workspace is None and stream is None:
        done = (_fast_calls or _bind_fast()).layer_norm_backward(dy, x, weight, mean, rstd)
        if done is not None:
            return done
    with _place(stream, x):
        _refuse_grad(dy, x, weight, mean, rstd)
        f32 = _torch().float32
        d = _norm_desc(x)
        rows, cols = d.rows, d.cols
        pt = _norm_params(x, cols, weight, None)
        _check_dense(dy, (rows, cols), x.dtype, x, "dy")
        _check_dense(mean, (rows,), f32, x, "mean")
        _check_dense(rstd, (rows,), f32, x, "rstd")
        pdt = weight.dtype if weight is not None else f32 if param_dtype is None else param_dtype
        dx = _torch().empty_like(dy)
        dweight, dbias = x.new_empty((2, cols), dtype=pdt).unbind(0)
        if weight is None:
            pt = _dtype_of(dweight, "param_dtype")
        ws = _scratch(workspace, iq_layer_norm_workspace_bytes(d), x)
        st = iq_layer_norm_backward(d, x.data_ptr(), dy.data_ptr(), _ptr(weight), pt, mean.data_ptr(), rstd.data_ptr(),
                                    dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), ws.data_ptr(), _stream_for(x))
        if st:
            _check(st, "iq_layer_norm_backward")
        return dx, dweight, dbias


def _gated_desc(x, w_gate, w_up, act: str):
    bf16 = _torch().bfloat16
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    if x.dim() != 2 or x.dtype != bf16 or not (x.is_contiguous() or x.shape[1] == 1 or x.stride(1) == 1):
        raise ValueError("x must be a 2-D bfloat16 tensor with unit column stride")
    tokens, cols = x.shape
    if w_gate.dim() != 2 or w_gate.shape[1] != cols:
        raise ValueError("w_gate must be [features, cols]")
    features = w_gate.shape[0]
    _check_dense(w_gate, (features, cols), bf16, x, "w_gate")
    _check_dense(w_up, (features, cols), bf16, x, "w_up")
    return IQGatedDesc(ACTS[act], IQ_BF16, tokens, cols, features, x.stride(0) if tokens > 1 and cols > 0 else cols, 0, 0)


def gated(x, w_gate, w_up, act: str = "silu", *, save: bool = False, out=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T) in one kernel, for BF16 x [tokens,
    cols] and weights [features, cols]; with save=True returns h and what
    gated_backward needs."""
    if out is None and stream is None and act in ACTS:
        done = (_fast_calls or _bind_fast()).gated(x, w_gate, w_up, ACTS[act], bool(save))
        if done is not None:
            return done
    with _place(stream, x):
        _refuse_grad(x, w_gate, w_up, out)
        d = _gated_desc(x, w_gate, w_up, act)
        h = _result(out, (d.tokens, d.features), x.dtype, x)
        saved = x.new_empty((2, d.tokens, d.features), dtype=_torch().float32) if save else None
        st = iq_gated_forward(d, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), h.data_ptr(), _ptr(saved),
                              _stream_for(x))
        if st:
            _check(st, "iq_gated_forward")
        return (h, saved) if save else h


def gated_backward(dh, x, w_gate, w_up, saved, act: str = "silu", *, workspace=None, stream=None):
    """Gradients of gated from dh [tokens, features] and the forward pass's
    saved values: dx, dw_gate and dw_up, BF16."""
    if workspace is None and stream is None and act in ACTS:
        done = (_fast_calls or _bind_fast()).gated_backward(dh, x, w_gate, w_up, saved, ACTS[act])
        if done is not None:
            return done
    with _place(stream, x):
        _refuse_grad(dh, x, w_gate, w_up, saved)
        d = _gated_desc(x, w_gate, w_up, act)
        tokens, cols, features = d.tokens, d.cols, d.features
        _check_dense(dh, (tokens, features), x.dtype, x, "dh")
        _check_dense(saved, (2, tokens, features), _torch().float32, x, "saved")
        dx = x.new_empty((tokens, cols))
        dwg, dwu = x.new_empty((2, features, cols)).unbind(0)
        ws = _scratch(workspace, iq_gated_workspace_bytes(d), x)
        st = iq_gated_backward(d, dh.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), saved.data_ptr(),
                               dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), ws.data_ptr(), _stream_for(x))
        if st:
            _check(st, "iq_gated_backward")
        return dx, dwg, dwu


# format -> codes and elements per scale, bytes per scale
_PACKED = {"int4": (128, 2), "nvfp4": (16, 1), "mxfp4": (32, 1)}


def _packed_f32(out_dtype):
    """Whether the result is float32 (not bfloat16); None for any other type."""
    code = IQ_BF16 if out_dtype is None else _dtypes().get(out_dtype)
    return None if code is None else code == IQ_F32


def _packed_x(x, cols: int):
    if x.dim() != 2 or x.shape[1] != cols or x.dtype != _torch().bfloat16 or not x.is_contiguous():
        raise ValueError("x must be a contiguous BF16 [n1, K] tensor")


def _packed_weights(q: "Quantized", x, what: str = "weights"):
    """Checks of packed weights; the addresses of their codes, scales and global scale."""
    if q.fmt not in _PACKED:
        raise ValueError(f"{what} must be INT4, NVFP4 or MXFP4")
    group, size = _PACKED[q.fmt]
    codes, scales, uint8 = q.codes, q.scales, _torch().uint8
    if codes.dtype is not uint8 or codes.get_device() != x.get_device() or not codes.is_contiguous() or codes.numel() < q.rows * (q.cols // 2):
        _check_buffer(codes, q.rows * (q.cols // 2), f"{what}' codes", x.device, uint8)
    if (scales.get_device() != x.get_device() or not scales.is_contiguous()
            or scales.numel() * scales.element_size() < q.rows * (q.cols // group) * size):
        _check_buffer(scales, q.rows * (q.cols // group) * size, f"{what}' scales", x.device)
    if q.fmt == "nvfp4":
        _check_buffer(q.global_scale, 4, f"{what}' global_scale", x.device, _torch().float32)
    return codes.data_ptr(), scales.data_ptr(), _ptr(q.global_scale)


def packed_gemv(q: "Quantized", x, out_dtype=None, out=None, stream=None):
    """z[t, j] = sum_k x[t, k] w[j, k] for 1 to 64 BF16 tokens x [n1, K] and
    INT4, NVFP4 or MXFP4 weights q [N0, K] (from quantize); z [n1, N0] is
    bfloat16 (by default) or float32, token-major."""
    rows, cols = q.rows, q.cols
    f32 = _packed_f32(out_dtype)
    if out is None and stream is None and f32 is not None and q.fmt in _PACKED:
        done = (_fast_calls or _bind_fast()).packed_gemv(x, FORMATS[q.fmt], rows, cols, f32, q.codes, q.scales, q.global_scale)
        if done is not None:
            return done
    with _place(stream, x):
        _refuse_grad(x, out)
        _packed_x(x, cols)
        codes, scales, gscale = _packed_weights(q, x)
        n1 = x.shape[0]
        z = _result(out, (n1, rows), x.dtype if out_dtype is None else out_dtype, x)
        st = iq_packed_gemv(make_desc(q.fmt, "block", rows, cols), codes, scales, gscale, x.data_ptr(), IQ_BF16, n1,
                            z.data_ptr(), _dtype_of(z, "out"), _stream_for(x))
        if st:
            _check(st, "iq_packed_gemv")
        return z


def packed_gated(q_gate: "Quantized", q_up: "Quantized", x, act: str = "silu", out_dtype=None, out=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T) for 1 to 64 BF16 tokens with both
    weights packed in the same format, in one launch; h [n1, N0] is bfloat16
    (by default) or float32."""
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    rows, cols = q_gate.rows, q_gate.cols
    if q_gate.fmt != q_up.fmt or rows != q_up.rows or cols != q_up.cols:
        raise ValueError("gate and up weights disagree on format or shape")
    f32 = _packed_f32(out_dtype)
    if out is None and stream is None and f32 is not None and q_gate.fmt in _PACKED:
        done = (_fast_calls or _bind_fast()).packed_gated(x, FORMATS[q_gate.fmt], rows, cols, f32, ACTS[act], q_gate.codes, q_gate.scales,
                                                     q_gate.global_scale, q_up.codes, q_up.scales, q_up.global_scale)
        if done is not None:
            return done
    with _place(stream, x):
        _refuse_grad(x, out)
        _packed_x(x, cols)
        gate, up = _packed_weights(q_gate, x, "gate weights"), _packed_weights(q_up, x, "up weights")
        n1 = x.shape[0]
        h = _result(out, (n1, rows), x.dtype if out_dtype is None else out_dtype, x)
        st = iq_packed_gated(make_desc(q_gate.fmt, "block", rows, cols), ACTS[act], *gate, *up, x.data_ptr(), IQ_BF16, n1,
                             h.data_ptr(), _dtype_of(h, "out"), _stream_for(x))
        if st:
            _check(st, "iq_packed_gated")
        return h
