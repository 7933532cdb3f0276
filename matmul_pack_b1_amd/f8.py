"""8-bit block-scaled matrices and their product: ctypes binding over the
entry points of include/hyb_f8.h.

    Q = f8.pack(w)          # weight, n x k: one scale per 128 x 128 block
    y = f8.gemm(Q, x)       # y = x Q^T, x quantised per 1 x 128 block in the call
    X = f8.quant(x)         # quantise once for several products
    y = f8.gemm(Q, X)
    w8 = f8.unpack(Q)       # the values the codes stand for

Argument marshalling only, as in binding.py: torch tensors supply device
memory and the current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from functools import lru_cache

import torch

from . import binding as hb

WEIGHT, ROWS = 1, 2   # HYB_F8_WEIGHT, HYB_F8_ROWS
EXPORTED = ("hyb_f8_size", "hyb_f8_quantize", "hyb_f8_dequantize", "hyb_f8_gemm_workspace_size", "hyb_f8_gemm",
            "hyb_f8_linear_workspace_size", "hyb_f8_linear")
KIND_NAMES = {WEIGHT: "weight", ROWS: "rows"}


class HybF8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_ready = False


def lib() -> ctypes.CDLL:
    global _ready
    L = hb.lib()
    if not _ready:
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        SZ, M = ctypes.c_size_t, ctypes.POINTER(HybF8)
        L.hyb_f8_size.argtypes = [I64, I64, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
        L.hyb_f8_quantize.argtypes = [P, I32, I64, I64, I64, I32, M, P]
        L.hyb_f8_dequantize.argtypes = [M, I64, I64, P, I32, I64, P]
        L.hyb_f8_gemm_workspace_size.argtypes = [I64, I64, I32, ctypes.POINTER(SZ)]
        L.hyb_f8_gemm.argtypes = [M, I64, I64, M, I32, P, I32, I64, P, SZ, P]
        L.hyb_f8_linear_workspace_size.argtypes = [I64, I64, I32, ctypes.POINTER(SZ)]
        L.hyb_f8_linear.argtypes = [M, I64, I64, P, I32, I32, I64, P, I32, I64, P, SZ, P]
        for name in EXPORTED:
            getattr(L, name).restype = I32
        _ready = True
    return L


_CODES = {torch.float16: hb.HYB_F16, torch.bfloat16: hb.HYB_BF16, torch.float32: hb.HYB_F32}


def _code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}: float16, bfloat16 or float32")
    return code


def _on(device):
    """Makes `device` current for a call (a decode step's calls are short: no
    switch where it is already)."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


# torch's current-stream handle without building a Stream object (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    return _raw_stream(device.index) if _raw_stream else hb._stream(device)


def _pitch(t, k) -> int:
    """Row stride of a 2-D tensor (k where it has at most one row)."""
    return int(t.stride(0)) if t.numel() and t.shape[0] > 1 else int(k)


def sizes(rows: int, k: int) -> tuple[int, int]:
    """Bytes of the codes and of the scales of a rows x k matrix."""
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    hb.check(lib().hyb_f8_size(int(rows), int(k), ctypes.byref(a), ctypes.byref(b)), "hyb_f8_size")
    return int(a.value), int(b.value)


@lru_cache(maxsize=4096)
def _sizes(rows, k):
    return sizes(rows, k)


@lru_cache(maxsize=4096)
def _ws_bytes(linear, n, k, m, index):
    """Workspace bytes of a product on device `index` (a function of the shape
    and the device's compute units)."""
    nbytes = ctypes.c_size_t(0)
    name = "hyb_f8_linear_workspace_size" if linear else "hyb_f8_gemm_workspace_size"
    hb.check(getattr(lib(), name)(n, k, m, ctypes.byref(nbytes)), name)
    return int(nbytes.value)


@dataclass
class F8Matrix:
    """A quantised matrix: kind WEIGHT or ROWS, its shape, the dtype it was
    made from, and two device buffers."""
    kind: int
    shape: tuple
    dtype: object
    codes: object
    scales: object

    @property
    def device(self):
        return self.codes.device

    def struct(self) -> HybF8:
        return HybF8(hb._ptr(self.codes), hb._ptr(self.scales))

    def weight_bytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _check_matrix(Q, kind, name):
    if not isinstance(Q, F8Matrix):
        raise TypeError(f"{name} must be an F8Matrix")
    if Q.kind != kind:
        raise TypeError(f"{name} is quantised as {KIND_NAMES[Q.kind]}, expected {KIND_NAMES[kind]}")
    codes, scales, need = Q.codes, Q.scales, _sizes(*Q.shape)
    if (codes.numel(), scales.numel()) != need:
        raise ValueError(f"{name}: buffers of {(codes.numel(), scales.numel())} bytes, its shape needs {need}")
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise TypeError(f"{name}: buffers of {codes.dtype} and {scales.dtype}, expected uint8")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: buffers must be contiguous")
    if scales.device != codes.device:
        raise ValueError(f"{name}: its scales are on {scales.device}, its codes on {codes.device}")


def _quantize(a, kind, out, name):
    hb._check_2d(a, name)
    code = _code(a.dtype)
    rows, k = a.shape
    nc, ns = _sizes(rows, k)
    if out is not None:
        _check_matrix(out, kind, "out")
        if tuple(out.shape) != (rows, k):
            raise ValueError(f"out is {tuple(out.shape)}, expected {(rows, k)}")
    hb._check_gpu(a, name)
    if out is None:
        out = F8Matrix(kind, (rows, k), a.dtype, torch.empty(nc, dtype=torch.uint8, device=a.device),
                       torch.empty(ns, dtype=torch.uint8, device=a.device))
    else:
        if out.codes.device != a.device:
            raise ValueError(f"out is on {out.codes.device}, {name} on {a.device}")
        out.dtype = a.dtype
    with _on(a.device):
        hb.check(lib().hyb_f8_quantize(hb._ptr(a), code, rows, k, _pitch(a, k), kind, out.struct(),
                                       _stream(a.device)), "hyb_f8_quantize")
    return out


def pack(w, out: F8Matrix | None = None) -> F8Matrix:
    """Quantise a weight (n x k; float16, bfloat16 or float32; unit column
    stride) with one scale per 128 x 128 block.  `out` reuses buffers."""
    return _quantize(w, WEIGHT, out, "w")


def quant(x, out: F8Matrix | None = None) -> F8Matrix:
    """Quantise activations (m x k) with one scale per 1 x 128 block, once for
    every product that reads them."""
    return _quantize(x, ROWS, out, "x")


def unpack(Q: F8Matrix, out_dtype=None, out=None):
    """The values the codes of Q stand for (default dtype: that of the matrix
    it was made from, which holds them exactly)."""
    if not isinstance(Q, F8Matrix):
        raise TypeError("Q must be an F8Matrix")
    _check_matrix(Q, Q.kind, "Q")
    rows, k = Q.shape
    if out is not None and out_dtype is None:
        out_dtype = out.dtype
    tdt = out_dtype if out_dtype is not None else Q.dtype
    code = _code(tdt)
    if out is None:
        out = torch.empty((rows, k), dtype=tdt, device=Q.device)
    hb._check_out(out, (rows, k), tdt)
    hb._check_gpu(out, "out", Q.device)
    with _on(Q.device):
        hb.check(lib().hyb_f8_dequantize(Q.struct(), rows, k, hb._ptr(out), code, _pitch(out, k),
                                         _stream(Q.device)), "hyb_f8_dequantize")
    return out


def workspace_bytes(Q: F8Matrix, m: int, quantised: bool = False) -> int:
    """Workspace bytes of gemm() for m tokens on the current device; with
    `quantised`, for activations that quant() gave."""
    return _ws_bytes(not quantised, Q.shape[0], Q.shape[1], int(m), torch.cuda.current_device()
                     if torch.cuda.is_available() else -1)


def gemm(Q: F8Matrix, x, out_dtype=None, out=None, workspace=None):
    """Y = X Q^T for any number of tokens (fp32 by default, or float16 /
    bfloat16).  x: activations (m x k; quantised here, for this call) or what
    quant() gave.  The workspace comes from torch's allocator unless
    `workspace` (a contiguous device tensor of at least workspace_bytes(Q, m)
    bytes) is given."""
    _check_matrix(Q, WEIGHT, "Q")
    n, k = Q.shape
    quantised = isinstance(x, F8Matrix)
    if quantised:
        _check_matrix(x, ROWS, "x")
    else:
        hb._check_2d(x, "x")
        xcode = _code(x.dtype)
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns, the weight has k = {k}")
    m = x.shape[0]
    if out is not None and out_dtype is None:
        out_dtype = out.dtype
    tdt = out_dtype if out_dtype is not None else torch.float32
    code = _code(tdt)
    device = Q.codes.device
    if out is not None:
        hb._check_out(out, (m, n), tdt)
    if quantised:
        if x.device != device:
            raise ValueError(f"x is on {x.device}, Q on {device}")
    else:
        hb._check_gpu(x, "x", device)
    if out is None:
        out = torch.empty((m, n), dtype=tdt, device=device)
    hb._check_gpu(out, "out", device)
    with _on(device):
        if workspace is None:
            nbytes = _ws_bytes(not quantised, n, k, m, device.index)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        else:
            hb._check_gpu(workspace, "workspace", device)
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
            nbytes = workspace.numel() * workspace.element_size()
        ws, stream = hb._ptr(workspace), _stream(device)
        if quantised:
            st = lib().hyb_f8_gemm(Q.struct(), n, k, x.struct(), m, hb._ptr(out), code, _pitch(out, n), ws, nbytes, stream)
        else:
            st = lib().hyb_f8_linear(Q.struct(), n, k, hb._ptr(x), xcode, m, _pitch(x, k), hb._ptr(out), code,
                                     _pitch(out, n), ws, nbytes, stream)
    if st:
        hb.check(st, "hyb_f8_gemm" if quantised else "hyb_f8_linear")
    return out
