"""4-bit weights with group scales and their product: ctypes binding over the
entry points of include/hyb_q4.h.

    Q = q4.pack(w)          # n x k: e2m1 codes, one power-of-two scale per 32 columns of a row
    y = q4.gemm(Q, x)       # y = x Q^T, x in 16 bits, any number of tokens
    w4 = q4.unpack(Q)       # the values the codes stand for

Argument marshalling only, as in binding.py: torch tensors supply device
memory and the current stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from functools import lru_cache

import torch

from . import binding as hb
from .f8 import _code, _on, _pitch, _stream

EXPORTED = ("hyb_q4_size", "hyb_q4_quantize", "hyb_q4_dequantize", "hyb_q4_gemm_workspace_size", "hyb_q4_gemm")


class HybQ4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_ready = False


def lib() -> ctypes.CDLL:
    global _ready
    L = hb.lib()
    if not _ready:
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        SZ, M = ctypes.c_size_t, ctypes.POINTER(HybQ4)
        L.hyb_q4_size.argtypes = [I64, I64, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
        L.hyb_q4_quantize.argtypes = [P, I32, I64, I64, I64, M, P]
        L.hyb_q4_dequantize.argtypes = [M, I64, I64, P, I32, I64, P]
        L.hyb_q4_gemm_workspace_size.argtypes = [I64, I64, I32, ctypes.POINTER(SZ)]
        L.hyb_q4_gemm.argtypes = [M, I64, I64, P, I32, I32, I64, P, I32, I64, P, SZ, P]
        for name in EXPORTED:
            getattr(L, name).restype = I32
        _ready = True
    return L


def sizes(n: int, k: int) -> tuple[int, int]:
    """Bytes of the codes and of the scales of an n x k weight."""
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    hb.check(lib().hyb_q4_size(int(n), int(k), ctypes.byref(a), ctypes.byref(b)), "hyb_q4_size")
    return int(a.value), int(b.value)


@lru_cache(maxsize=4096)
def _sizes(n, k):
    return sizes(n, k)


@lru_cache(maxsize=4096)
def _ws_bytes(n, k, m, index):
    """Workspace bytes of a product on device `index` (a function of the shape
    and the device's compute units)."""
    nbytes = ctypes.c_size_t(0)
    hb.check(lib().hyb_q4_gemm_workspace_size(n, k, m, ctypes.byref(nbytes)), "hyb_q4_gemm_workspace_size")
    return int(nbytes.value)


@dataclass
class Q4Matrix:
    """A 4-bit weight: its shape, the dtype it was made from, and two device
    buffers."""
    shape: tuple
    dtype: object
    codes: object
    scales: object

    @property
    def device(self):
        return self.codes.device

    def struct(self) -> HybQ4:
        return HybQ4(hb._ptr(self.codes), hb._ptr(self.scales))

    def weight_bytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _check_matrix(Q, name):
    if not isinstance(Q, Q4Matrix):
        raise TypeError(f"{name} must be a Q4Matrix")
    codes, scales, need = Q.codes, Q.scales, _sizes(*Q.shape)
    if (codes.numel(), scales.numel()) != need:
        raise ValueError(f"{name}: buffers of {(codes.numel(), scales.numel())} bytes, its shape needs {need}")
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise TypeError(f"{name}: buffers of {codes.dtype} and {scales.dtype}, expected uint8")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: buffers must be contiguous")
    if scales.device != codes.device:
        raise ValueError(f"{name}: its scales are on {scales.device}, its codes on {codes.device}")


def pack(w, out: Q4Matrix | None = None) -> Q4Matrix:
    """Quantise a weight (n x k; float16, bfloat16 or float32; unit column
    stride).  `out` reuses buffers."""
    hb._check_2d(w, "w")
    code = _code(w.dtype)
    n, k = w.shape
    nc, ns = _sizes(n, k)
    if out is not None:
        _check_matrix(out, "out")
        if tuple(out.shape) != (n, k):
            raise ValueError(f"out is {tuple(out.shape)}, expected {(n, k)}")
    hb._check_gpu(w, "w")
    if out is None:
        out = Q4Matrix((n, k), w.dtype, torch.empty(nc, dtype=torch.uint8, device=w.device),
                       torch.empty(ns, dtype=torch.uint8, device=w.device))
    else:
        if out.codes.device != w.device:
            raise ValueError(f"out is on {out.codes.device}, w on {w.device}")
        out.dtype = w.dtype
    with _on(w.device):
        hb.check(lib().hyb_q4_quantize(hb._ptr(w), code, n, k, _pitch(w, k), out.struct(), _stream(w.device)),
                 "hyb_q4_quantize")
    return out


def unpack(Q: Q4Matrix, out_dtype=None, out=None):
    """The values the codes of Q stand for (default dtype: that of the matrix
    it was made from)."""
    _check_matrix(Q, "Q")
    n, k = Q.shape
    if out is not None and out_dtype is None:
        out_dtype = out.dtype
    tdt = out_dtype if out_dtype is not None else Q.dtype
    code = _code(tdt)
    if out is None:
        out = torch.empty((n, k), dtype=tdt, device=Q.device)
    hb._check_out(out, (n, k), tdt)
    hb._check_gpu(out, "out", Q.device)
    with _on(Q.device):
        hb.check(lib().hyb_q4_dequantize(Q.struct(), n, k, hb._ptr(out), code, _pitch(out, k), _stream(Q.device)),
                 "hyb_q4_dequantize")
    return out


def workspace_bytes(Q: Q4Matrix, m: int) -> int:
    """Workspace bytes of gemm() for m tokens on the current device."""
    return _ws_bytes(Q.shape[0], Q.shape[1], int(m),
                     torch.cuda.current_device() if torch.cuda.is_available() else -1)


def _workspace(workspace, need, device):
    """(tensor, bytes): the caller's workspace, or one from torch's allocator."""
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=device) if need else None), need
    hb._check_gpu(workspace, "workspace", device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def gemm(Q: Q4Matrix, x, out_dtype=None, out=None, workspace=None):
    """Y = X Q^T for any number of tokens (fp32 by default, or float16 /
    bfloat16).  x: activations, m x k, float16 or bfloat16.  The workspace comes
    from torch's allocator unless `workspace` (a contiguous device tensor of at
    least workspace_bytes(Q, m) bytes) is given."""
    _check_matrix(Q, "Q")
    n, k = Q.shape
    hb._check_2d(x, "x")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x is {x.dtype}, expected bfloat16 or float16")
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
    hb._check_gpu(x, "x", device)
    if out is None:
        out = torch.empty((m, n), dtype=tdt, device=device)
    hb._check_gpu(out, "out", device)
    with _on(device):
        ws, nbytes = _workspace(workspace, _ws_bytes(n, k, m, device.index) if workspace is None else 0, device)
        st = lib().hyb_q4_gemm(Q.struct(), n, k, hb._ptr(x), _code(x.dtype), m, _pitch(x, k), hb._ptr(out), code,
                               _pitch(out, n), hb._ptr(ws), nbytes, _stream(device))
    if st:
        hb.check(st, "hyb_q4_gemm")
    return out
