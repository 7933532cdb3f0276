"""Gated feed-forward projection and its gradients: ctypes binding over the
entry points of include/hyb_gated.h.

    h = gated.forward(G, U, x)                         # act(x G^T) * (x U^T)
    h, g, u = gated.forward(G, U, x, save=True)        # keeps what the gradients need
    dx, dg, du = gated.backward(G, U, x, g, u, dh, need_dw=True)

G and U are two PackedWeight (binding.py) of one shape, or two Q4Matrix (q4.py;
no gradients).  Argument marshalling only, as in binding.py.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as hb
from . import q4
from .f8 import _code, _on, _pitch, _stream

ACTS = {"silu": 1, "gelu": 2, "gelu_tanh": 3}   # HYB_ACT_*
DX, DW = 1, 2                                    # HYB_GATED_DX, HYB_GATED_DW
EXPORTED = ("hyb_gated_workspace_size", "hyb_gated", "hyb_gated_backward")


class HybGatedPair(ctypes.Structure):
    _fields_ = [("gate_layout", ctypes.POINTER(hb.HybLayout)), ("gate", ctypes.POINTER(hb.HybPacked)),
                ("up_layout", ctypes.POINTER(hb.HybLayout)), ("up", ctypes.POINTER(hb.HybPacked)),
                ("gate4", ctypes.POINTER(q4.HybQ4)), ("up4", ctypes.POINTER(q4.HybQ4)),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


_ready = False


def lib() -> ctypes.CDLL:
    global _ready
    L = q4.lib()
    if not _ready:
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        W = ctypes.POINTER(HybGatedPair)
        L.hyb_gated_workspace_size.argtypes = [W, I32, I32, ctypes.POINTER(SZ)]
        L.hyb_gated.argtypes = [W, I32, P, I32, I32, I64, P, I64, P, I64, P, I64, P, SZ, P]
        L.hyb_gated_backward.argtypes = [W, I32, P, I32, I32, I64, P, I64, P, I64, P, I64, P, I64, P, I64, P, I64, P, SZ,
                                         P]
        for name in EXPORTED:
            getattr(L, name).restype = I32
        _ready = True
    return L


def _pair(G, U):
    """(C pair, n, k); the ctypes objects stay alive with the pair."""
    if isinstance(G, hb.PackedWeight) and isinstance(U, hb.PackedWeight):
        if tuple(G.shape) != tuple(U.shape):
            raise ValueError(f"gate is {tuple(G.shape)}, up {tuple(U.shape)}")
        if G.dtype != U.dtype:
            raise TypeError(f"gate is {G.dtype}, up {U.dtype}")
        n, k = G.shape
        return HybGatedPair(ctypes.pointer(G.layout), ctypes.pointer(G.packed_struct()), ctypes.pointer(U.layout),
                            ctypes.pointer(U.packed_struct()), None, None, n, k), n, k
    if not (isinstance(G, q4.Q4Matrix) and isinstance(U, q4.Q4Matrix)):
        raise TypeError("the weights must be two PackedWeight or two Q4Matrix")
    q4._check_matrix(G, "gate")
    q4._check_matrix(U, "up")
    if tuple(G.shape) != tuple(U.shape):
        raise ValueError(f"gate is {tuple(G.shape)}, up {tuple(U.shape)}")
    n, k = G.shape
    return HybGatedPair(None, None, None, None, ctypes.pointer(G.struct()), ctypes.pointer(U.struct()), n, k), n, k


def _check(G, U, x, act):
    pair, n, k = _pair(G, U)
    if act not in ACTS:
        raise ValueError(f"act is {act!r}, expected one of {', '.join(ACTS)}")
    hb._check_2d(x, "x")
    if isinstance(G, hb.PackedWeight):
        hb._check_x(G, x)
    elif x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x is {x.dtype}, expected bfloat16 or float16")
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns, the weights have k = {k}")
    return pair, n, k, x.shape[0]


def _check_devices(G, U, x):
    hb._check_gpu(x, "x", G.device)
    for W in (G, U):
        if isinstance(W, hb.PackedWeight):
            hb._check_same_device(W, x.device)
        elif W.device != x.device:
            raise ValueError(f"a weight is on {W.device}, x on {x.device}")


def _need(pair, m, what):
    nbytes = ctypes.c_size_t(0)
    hb.check(lib().hyb_gated_workspace_size(ctypes.byref(pair), m, what, ctypes.byref(nbytes)),
             "hyb_gated_workspace_size")
    return int(nbytes.value)


def workspace_bytes(G, U, m: int, dx: bool = False, dw: bool = False) -> int:
    """Workspace bytes of forward() (neither flag) or backward() on the current
    device."""
    return _need(_pair(G, U)[0], int(m), (DX if dx else 0) | (DW if dw else 0))


def forward(G, U, x, act="silu", save=False, out=None, workspace=None):
    """H = act(x G^T) * (x U^T) for any number of tokens, of x's dtype (packed
    weights: their own; 4-bit ones: float16 or bfloat16).  act: "silu", "gelu" or
    "gelu_tanh".  With `save` (packed weights) the result is (H, x G^T, x U^T), the
    last two in float32, for backward().  `out` may give H.  The workspace
    comes from torch's allocator unless `workspace` (a contiguous device tensor
    of at least workspace_bytes(G, U, m) bytes) is given."""
    pair, n, k, m = _check(G, U, x, act)
    if save and not isinstance(G, hb.PackedWeight):
        raise TypeError("4-bit weights have no gradients")
    if out is not None:
        hb._check_out(out, (m, n), x.dtype)
    _check_devices(G, U, x)
    h = torch.empty((m, n), dtype=x.dtype, device=x.device) if out is None else out
    hb._check_gpu(h, "out", x.device)
    g, u = (torch.empty((m, n), dtype=torch.float32, device=x.device) for _ in range(2)) if save else (None, None)
    with _on(x.device):
        ws, nbytes = q4._workspace(workspace, _need(pair, m, 0) if workspace is None else 0, x.device)
        hb.check(lib().hyb_gated(ctypes.byref(pair), ACTS[act], hb._ptr(x), _code(x.dtype), m, _pitch(x, k), hb._ptr(h),
                                 _pitch(h, n), hb._ptr(g), n, hb._ptr(u), n, hb._ptr(ws), nbytes, _stream(x.device)),
                 "hyb_gated")
    return (h, g, u) if save else h


def backward(G, U, x, g, u, dh, act="silu", need_dx=True, need_dw=False, dx=None, dw_gate=None, dw_up=None,
             workspace=None):
    """(dx, dw_gate, dw_up) for the gradient `dh` (m x n, x's dtype) of H; g and
    u are what forward(save=True) gave for the same weights, x and act.  dx is
    m x k; the weights' gradients n x k and dense: every entry's, dropped ones
    included.  What is not asked for is None; `dx`, `dw_gate` and `dw_up` may
    give the outputs."""
    pair, n, k, m = _check(G, U, x, act)
    if not isinstance(G, hb.PackedWeight):
        raise TypeError("4-bit weights have no gradients")
    for t, dtype, name in ((g, torch.float32, "g"), (u, torch.float32, "u"), (dh, x.dtype, "dh")):
        hb._check_out(t, (m, n), dtype, name)
    if (dw_gate is None) != (dw_up is None):
        raise ValueError("give both dw_gate and dw_up, or neither")
    need_dx, need_dw = need_dx or dx is not None, need_dw or dw_gate is not None
    for t, shape, name in ((dx, (m, k), "dx"), (dw_gate, (n, k), "dw_gate"), (dw_up, (n, k), "dw_up")):
        if t is not None:
            hb._check_out(t, shape, x.dtype, name)
    _check_devices(G, U, x)
    new = lambda rows: torch.empty((rows, k), dtype=x.dtype, device=x.device)  # noqa: E731
    if need_dx and dx is None:
        dx = new(m)
    if need_dw and dw_gate is None:
        dw_gate, dw_up = new(n), new(n)
    for t, name in ((g, "g"), (u, "u"), (dh, "dh"), (dx, "dx"), (dw_gate, "dw_gate"), (dw_up, "dw_up")):
        if t is not None:
            hb._check_gpu(t, name, x.device)
    if not need_dx and not need_dw:
        return None, None, None
    with _on(x.device):
        what = (DX if need_dx else 0) | (DW if need_dw else 0)
        ws, nbytes = q4._workspace(workspace, _need(pair, m, what) if workspace is None else 0, x.device)
        hb.check(lib().hyb_gated_backward(
            ctypes.byref(pair), ACTS[act], hb._ptr(x), _code(x.dtype), m, _pitch(x, k), hb._ptr(g), _pitch(g, n),
            hb._ptr(u), _pitch(u, n), hb._ptr(dh), _pitch(dh, n), hb._ptr(dx), _pitch(dx, k) if need_dx else 0,
            hb._ptr(dw_gate), _pitch(dw_gate, k) if need_dw else 0, hb._ptr(dw_up), _pitch(dw_up, k) if need_dw else 0,
            hb._ptr(ws), nbytes, _stream(x.device)), "hyb_gated_backward")
    return dx, dw_gate, dw_up
