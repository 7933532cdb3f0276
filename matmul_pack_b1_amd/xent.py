"""Softmax cross entropy over a vocabulary projection, without the logits in
memory: ctypes binding over the entry points of include/hyb_xent.h.

    P = hb.pack(w, tile_map, 128, 128)            # or f8.pack(w)
    loss, lse = xent.loss(P, x, target)           # per token, fp32
    dx, dw = xent.backward(P, x, target, lse, grad)

The head P is a PackedWeight (binding.py) or an F8Matrix weight (f8.py); an
8-bit head has no weight gradient.  Argument marshalling only, as in
binding.py.
"""
from __future__ import annotations

import ctypes

from . import binding as hb
from . import f8

DX, DW = 1, 2   # HYB_XENT_DX, HYB_XENT_DW
EXPORTED = ("hyb_xent_workspace_size", "hyb_xent_piece_rows", "hyb_xent", "hyb_xent_backward")


class HybHead(ctypes.Structure):
    _fields_ = [("layout", ctypes.POINTER(hb.HybLayout)), ("packed", ctypes.POINTER(hb.HybPacked)),
                ("f8", ctypes.POINTER(f8.HybF8)), ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


_ready = False


def lib() -> ctypes.CDLL:
    global _ready
    L = f8.lib()
    if not _ready:
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        H = ctypes.POINTER(HybHead)
        L.hyb_xent_workspace_size.argtypes = [H, I32, I32, ctypes.POINTER(SZ)]
        L.hyb_xent_piece_rows.argtypes = [H, I32, I32, ctypes.POINTER(I64)]
        L.hyb_xent.argtypes = [H, I64, P, I32, I32, I64, P, I64, P, P, P, SZ, P]
        L.hyb_xent_backward.argtypes = [H, I64, P, I32, I32, I64, P, I64, P, P, P, I64, P, I64, P, SZ, P]
        for name in EXPORTED:
            getattr(L, name).restype = I32
        _ready = True
    return L


def _head(P):
    """(C head, n, k); the ctypes objects stay alive with the head."""
    if isinstance(P, hb.PackedWeight):
        n, k = P.shape
        return HybHead(ctypes.pointer(P.layout), ctypes.pointer(P.packed_struct()), None, n, k), n, k
    f8._check_matrix(P, f8.WEIGHT, "the head")
    n, k = P.shape
    return HybHead(None, None, ctypes.pointer(P.struct()), n, k), n, k


def _vector(t, m, dtype, name, device=None):
    if t.dim() != 1 or t.shape[0] != m:
        raise ValueError(f"{name} is {tuple(t.shape)}, expected ({m},)")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if m > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    if device is not None:
        hb._check_gpu(t, name, device)


def _check(P, x, target, n_vocab):
    torch = hb._torch()
    head, n, k = _head(P)
    hb._check_2d(x, "x")
    if isinstance(P, hb.PackedWeight):
        hb._check_x(P, x)
    elif x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x is {x.dtype}, expected bfloat16 or float16")
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns, the head has k = {k}")
    m = x.shape[0]
    _vector(target, m, torch.int64, "target")
    n_vocab = n if n_vocab is None else int(n_vocab)
    hb._check_gpu(x, "x", P.device)
    if isinstance(P, hb.PackedWeight):
        hb._check_same_device(P, x.device)
    hb._check_gpu(target, "target", x.device)
    return head, n, k, m, n_vocab


def workspace_bytes(P, m: int, dx: bool = False, dw: bool = False) -> int:
    """Workspace bytes of loss() (neither flag) or backward() on the current
    device."""
    return _need(_head(P)[0], int(m), dx, dw)


def piece_rows(P, m: int, dx: bool = False, dw: bool = False) -> int:
    """Rows of the head that loss() (neither flag) or backward() works through
    at a time for m tokens on the current device."""
    rows = ctypes.c_int64(0)
    hb.check(lib().hyb_xent_piece_rows(ctypes.byref(_head(P)[0]), int(m), (DX if dx else 0) | (DW if dw else 0),
                                       ctypes.byref(rows)), "hyb_xent_piece_rows")
    return int(rows.value)


def _need(head, m, dx, dw):
    nbytes = ctypes.c_size_t(0)
    hb.check(lib().hyb_xent_workspace_size(ctypes.byref(head), m, (DX if dx else 0) | (DW if dw else 0),
                                           ctypes.byref(nbytes)), "hyb_xent_workspace_size")
    return int(nbytes.value)


def _workspace(head, m, dx, dw, workspace, device):
    torch = hb._torch()
    if workspace is None:
        need = _need(head, m, dx, dw)
        return torch.empty(need, dtype=torch.uint8, device=device), need
    hb._check_gpu(workspace, "workspace", device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def loss(P, x, target, n_vocab=None, ignore_index=-100, workspace=None):
    """(loss, lse) per token, fp32.  x: hidden states (m x k, the packed
    head's dtype, or float16 / bfloat16 with an 8-bit head), target: int64[m].
    Rows of the head from n_vocab on are padding.  The workspace comes from
    torch's allocator unless `workspace` (a contiguous device tensor of at
    least workspace_bytes(P, m) bytes) is given."""
    torch = hb._torch()
    head, n, k, m, n_vocab = _check(P, x, target, n_vocab)
    out = torch.empty(m, dtype=torch.float32, device=x.device)
    lse = torch.empty(m, dtype=torch.float32, device=x.device)
    with f8._on(x.device):
        ws, nbytes = _workspace(head, m, False, False, workspace, x.device)
        hb.check(lib().hyb_xent(ctypes.byref(head), n_vocab, hb._ptr(x), f8._code(x.dtype), m, f8._pitch(x, k),
                                hb._ptr(target), int(ignore_index), hb._ptr(out), hb._ptr(lse), hb._ptr(ws), nbytes,
                                f8._stream(x.device)), "hyb_xent")
    return out, lse


def backward(P, x, target, lse, grad, n_vocab=None, ignore_index=-100, need_dx=True, need_dw=False, dx=None, dw=None,
             workspace=None):
    """(dx, dw) for the gradient `grad` (fp32[m]) of each token's loss; lse is
    what loss() gave.  dx is m x k of x's dtype; dw (packed heads only) n x k of
    the head's dtype, dense: every entry's gradient, dropped ones included.
    What is not asked for is None; `dx` and `dw` may give the outputs."""
    torch = hb._torch()
    head, n, k, m, n_vocab = _check(P, x, target, n_vocab)
    _vector(lse, m, torch.float32, "lse", x.device)
    _vector(grad, m, torch.float32, "grad", x.device)
    need_dx, need_dw = need_dx or dx is not None, need_dw or dw is not None
    if need_dw and not isinstance(P, hb.PackedWeight):
        raise TypeError("an 8-bit head has no weight gradient")
    if need_dx and dx is None:
        dx = torch.empty((m, k), dtype=x.dtype, device=x.device)
    if need_dw and dw is None:
        dw = torch.empty((n, k), dtype=x.dtype, device=x.device)
    for t, shape, name in ((dx, (m, k), "dx"), (dw, (n, k), "dw")):
        if t is not None:
            hb._check_out(t, shape, x.dtype, name)
            hb._check_gpu(t, name, x.device)
    with f8._on(x.device):
        ws, nbytes = _workspace(head, m, need_dx, need_dw, workspace, x.device)
        hb.check(lib().hyb_xent_backward(
            ctypes.byref(head), n_vocab, hb._ptr(x), f8._code(x.dtype), m, f8._pitch(x, k), hb._ptr(target),
            int(ignore_index), hb._ptr(lse), hb._ptr(grad), hb._ptr(dx), f8._pitch(dx, k) if need_dx else 0,
            hb._ptr(dw), f8._pitch(dw, k) if need_dw else 0, hb._ptr(ws), nbytes, f8._stream(x.device)),
            "hyb_xent_backward")
    return dx, dw
