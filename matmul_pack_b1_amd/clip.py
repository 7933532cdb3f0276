"""The 2-norm over a list of tensors and their scaling by it: ctypes binding
over the entry points of include/hyb_clip.h.

    norm = clip.norm(grads)              # fp32, on the device
    norm = clip.clip(grads, 1.0)         # the same, and grads scaled to a norm of at most 1

Argument marshalling only, as in binding.py.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import binding as hb
from .f8 import _CODES, _on, _stream

EXPORTED = ("hyb_clip_workspace_size", "hyb_norm", "hyb_clip")


class HybTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("lda", ctypes.c_int64), ("ldo", ctypes.c_int64), ("dtype", ctypes.c_int32)]


# One descriptor as the binding packs it (its last word is the type and padding).
_WORDS = 7
assert ctypes.sizeof(HybTensor) == 8 * _WORDS
_PER_LAUNCH = 64            # tensors of one launch, and the partial sums of one
_SUM_BYTES = 2048 * 8

_ready = False


def lib() -> ctypes.CDLL:
    global _ready
    L = hb.lib()
    if not _ready:
        P, I64, SZ, T = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
        L.hyb_clip_workspace_size.argtypes = [I64, T, ctypes.POINTER(SZ)]
        L.hyb_norm.argtypes = [I64, T, P, P, SZ, P]
        L.hyb_clip.argtypes = [I64, T, ctypes.c_float, P, P, SZ, P]
        for name in EXPORTED:
            getattr(L, name).restype = ctypes.c_int32
        _ready = True
    return L


def _rows(t, name):
    """(rows, columns, row stride) of a tensor that is contiguous, or 2-D with
    unit column stride and rows apart."""
    if t.is_contiguous():
        n = t.numel()
        return 1, n, n
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
        return t.shape[0], t.shape[1], t.stride(0)
    raise ValueError(f"{name} must be contiguous, or 2-D with unit column stride")


def _refuse(i, t, out, index):
    """What is wrong with a tensor and its output, of which something is."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"tensor {i} is a {type(t).__name__}")
    if t.dtype not in _CODES:
        raise TypeError(f"tensor {i} is {t.dtype}: float16, bfloat16 or float32")
    _rows(t, f"tensor {i}")
    if not isinstance(out, torch.Tensor) or out.shape != t.shape:
        raise ValueError(f"outs[{i}] must be a tensor of shape {tuple(t.shape)}")
    if out.dtype != t.dtype:
        raise TypeError(f"outs[{i}] is {out.dtype}, expected {t.dtype}")
    _rows(out, f"outs[{i}]")
    device = None if index is None else torch.device("cuda", index)
    hb._check_gpu(t, f"tensor {i}", device)
    hb._check_gpu(out, f"outs[{i}]", t.device)
    raise ValueError(f"tensor {i} cannot be used")


def _list(tensors, outs):
    """(count, C array as bytes, device).  The checks of each tensor come first
    in one condition (a step has many tensors, and its time is the host's)."""
    tensors = list(tensors)
    outs = tensors if outs is None else list(outs)
    if len(outs) != len(tensors):
        raise ValueError(f"{len(outs)} outs for {len(tensors)} tensors")
    words, index, Tensor = [], None, torch.Tensor
    for i, t in enumerate(tensors):
        out = outs[i]
        code = _CODES.get(t.dtype) if isinstance(t, Tensor) else None
        if code is None:
            _refuse(i, t, out, index)
        at = t.get_device()
        if at < 0 or (at != index and index is not None):
            _refuse(i, t, out, index)
        index = at
        if out is not t and (not isinstance(out, Tensor) or out.dtype is not t.dtype or out.shape != t.shape
                             or out.get_device() != at):
            _refuse(i, t, out, index)
        if t.is_contiguous() and (out is t or out.is_contiguous()):
            n = t.numel()
            words += (t.data_ptr(), out.data_ptr(), 1, n, n, n, code)
            continue
        rows, cols, lda = _rows(t, f"tensor {i}")
        orows, _, ldo = _rows(out, f"outs[{i}]")
        if orows != rows:   # one of the two is contiguous: take it as rows too
            rows, cols = t.shape
            lda, ldo = (s.stride(0) if not s.is_contiguous() else cols for s in (t, out))
        words += (t.data_ptr(), out.data_ptr(), rows, cols, lda, ldo, code)
    return (len(tensors), struct.pack(f"<{len(words)}Q", *words),
            None if index is None else torch.device("cuda", index))


def _run(tensors, outs, max_norm, out, workspace):
    count, array, device = _list(tensors, outs)
    if device is None:
        device = out.device if out is not None else torch.device("cuda", torch.cuda.current_device())
    if out is not None:
        if out.numel() != 1 or out.dtype != torch.float32:
            raise ValueError("out must hold one float32")
        hb._check_gpu(out, "out", device)
    with _on(device):
        if workspace is None:   # the most that so many tensors need
            nbytes = -(-count // _PER_LAUNCH) * _SUM_BYTES
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        else:
            hb._check_gpu(workspace, "workspace", device)
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
            nbytes = workspace.numel() * workspace.element_size()
        if out is None:
            out = torch.empty((), dtype=torch.float32, device=device)
        ws, stream = hb._ptr(workspace), _stream(device)
        if max_norm is None:
            hb.check(lib().hyb_norm(count, array, out.data_ptr(), ws, nbytes, stream), "hyb_norm")
        else:
            hb.check(lib().hyb_clip(count, array, float(max_norm), out.data_ptr(), ws, nbytes, stream), "hyb_clip")
    return out


def workspace_bytes(tensors, outs=None) -> int:
    """Workspace bytes of norm() or clip() of these tensors (and outs)."""
    count, array, _ = _list(tensors, outs)
    nbytes = ctypes.c_size_t(0)
    hb.check(lib().hyb_clip_workspace_size(count, array, ctypes.byref(nbytes)), "hyb_clip_workspace_size")
    return int(nbytes.value)


def norm(tensors, out=None, workspace=None):
    """The 2-norm over all elements of all tensors (float16, bfloat16 or float32,
    mixed as they come, on one GPU), an fp32 tensor of one element.  Each is
    contiguous, or 2-D with unit column stride.  The workspace comes from torch's
    allocator unless `workspace` (a contiguous device tensor of at least
    workspace_bytes(tensors, outs) bytes) is given."""
    return _run(tensors, None, None, out, workspace)


def clip(tensors, max_norm, outs=None, out=None, workspace=None):
    """norm(), and every tensor multiplied by min(1, max_norm / (norm + 1e-6)):
    in place, or into `outs` (tensors of the same shapes and dtypes)."""
    return _run(tensors, outs, max_norm, out, workspace)
