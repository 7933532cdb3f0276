"""The gated projection without a GPU: the oracle's gradients against
differences, the C ABI's refusals (include/hyb_gated.h) and workspace sizes, and
the binding's checks.  Every call below fails validation or does host work
only."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated, q4
from oracle import gated_oracle as go

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("act", list(gated.ACTS))
def test_oracle_gradients_against_differences(act):
    """The gradient of sum(dh * H) along random directions of x, W_g and W_u,
    against central differences: their own error is of the order of the step
    squared."""
    rng = np.random.default_rng(1)
    x, wg, wu, dh = (rng.standard_normal(s) for s in ((5, 7), (6, 7), (6, 7), (5, 6)))
    g, u, h = go.forward(x, wg, wu, act)
    dg, du = go.gradients(g, u, dh, act)
    grads = dg @ wg + du @ wu, dg.T @ x, du.T @ x
    step = 1e-5
    for i, grad in enumerate(grads):
        d = rng.standard_normal(grad.shape)
        at = [[x, wg, wu], [x, wg, wu]]
        for s, a in ((1, at[0]), (-1, at[1])):
            a[i] = a[i] + s * step * d
        diff = sum(s * (dh * go.forward(*a, act)[2]).sum() for s, a in ((1, at[0]), (-1, at[1]))) / (2 * step)
        assert abs(diff - (grad * d).sum()) <= 1e-6 * (1 + np.abs(grad * d).sum())


def test_oracle_activations_match_torch():
    g = torch.linspace(-9, 9, 1001, dtype=torch.float64)
    F = torch.nn.functional
    for act, f in (("silu", F.silu), ("gelu", F.gelu), ("gelu_tanh", lambda t: F.gelu(t, approximate="tanh"))):
        assert np.allclose(go.act(g.numpy(), act)[0], f(g).numpy(), rtol=1e-9, atol=1e-15)


def test_exports_match_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hyb_gated.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(hyb_[a-z0-9_]+)\s*\(", text))
    assert names == set(gated.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", hb.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (hyb_\w+)", out))


def _status(call):
    with pytest.raises(hb.HybError) as e:
        hb.check(call, "call")
    return e.value.status


P16 = 1 << 20  # any 16-byte aligned non-null address: never followed


def _layout(n=128, k=256, b1=64, b2=64, dtype="bf16", meta="idx2", sparse=1):
    return hb.plan(n, k, b1, b2, dtype, meta, np.arange(n // b1 * (k // b2)) % 2 * sparse)[0]


def _packed_pair(a=None, b=None, ga=(P16,) * 4, ub=(P16,) * 4):
    a, b = a or _layout(), b or _layout()
    p = gated.HybGatedPair(ctypes.pointer(a), ctypes.pointer(hb.HybPacked(*ga)), ctypes.pointer(b),
                           ctypes.pointer(hb.HybPacked(*ub)), None, None, 0, 0)
    p.keep = (a, b)
    return p


def _q4_pair(n=8, k=256, a=(P16, P16), b=(P16, P16)):
    return gated.HybGatedPair(None, None, None, None, ctypes.pointer(q4.HybQ4(*a)), ctypes.pointer(q4.HybQ4(*b)), n, k)


PAIRS = [
    (lambda: None, 1), (lambda: gated.HybGatedPair(), 1),
    (lambda: _packed_pair(b=_layout(n=192)), 2), (lambda: _packed_pair(b=_layout(k=320)), 2),
    (lambda: _packed_pair(b=_layout(dtype="f16")), 3), (lambda: _packed_pair(b=_layout(b1=128)), 4),
    (lambda: _packed_pair(b=_layout(meta="mask4")), 4), (lambda: _packed_pair(_layout(n=0), _layout(n=0)), 2),
    (lambda: _packed_pair(_layout(96, 256, 32), _layout(96, 256, 32)), 4),
    (lambda: _packed_pair(_layout(2 ** 21 + 256, 256, 256, 256), _layout(2 ** 21 + 256, 256, 256, 256)), 2),
    (lambda: _packed_pair(ga=(None, P16, P16, P16)), 1), (lambda: _packed_pair(ub=(P16, P16 + 8, P16, P16)), 1),
    (lambda: _packed_pair(ub=(P16, P16, P16, None)), 1),
    (lambda: _q4_pair(n=-1), 2), (lambda: _q4_pair(k=(1 << 22) + 1), 2), (lambda: _q4_pair(a=(None, P16)), 1),
    (lambda: _q4_pair(b=(P16, P16 + 4)), 1),
]


@pytest.mark.parametrize("make,status", PAIRS)
def test_refused_weights(make, status):
    pair = make()
    w = ctypes.byref(pair) if pair is not None else None
    L = gated.lib()
    st = L.hyb_gated(w, 1, P16, hb.HYB_BF16, 2, 2 ** 21, P16, 2 ** 22, None, 0, None, 0, P16, 1 << 60, None)
    assert _status(st) == status and hb.last_error()
    if pair is not None and pair.gate_layout:
        st = L.hyb_gated_backward(w, 1, P16, hb.HYB_BF16, 2, 2 ** 21, P16, 2 ** 22, P16, 2 ** 22, P16, 2 ** 22, P16,
                                  2 ** 22, None, 0, None, 0, P16, 1 << 60, None)
        assert _status(st) == status


def test_a_mixed_pair_is_refused():
    p = _packed_pair()
    p.gate4 = ctypes.pointer(q4.HybQ4(P16, P16))
    n = ctypes.c_size_t(0)
    assert _status(gated.lib().hyb_gated_workspace_size(ctypes.byref(p), 1, 0, ctypes.byref(n))) == 1
    p = _q4_pair()
    p.up4 = None
    assert _status(gated.lib().hyb_gated_workspace_size(ctypes.byref(p), 1, 0, ctypes.byref(n))) == 1


FORWARD = [
    (dict(act=0), 1), (dict(act=4), 1), (dict(dt=hb.HYB_F32), 3), (dict(dt=hb.HYB_F16), 3), (dict(m=-1), 2),
    (dict(m=(1 << 22) + 1), 2), (dict(x=None), 1), (dict(x=P16 + 8), 1), (dict(ldx=255), 1), (dict(ldx=260), 1),
    (dict(ldx=1 << 22), 4), (dict(h=None), 1), (dict(h=P16 + 1), 1), (dict(ldh=127), 1), (dict(ldh=2 ** 31 + 1), 4),
    (dict(g=None), 1), (dict(u=None), 1), (dict(g=P16 + 2), 1), (dict(ldu=100), 1), (dict(ws=None), 1),
    (dict(ws=P16 + 8), 1), (dict(nbytes=64), 1), (dict(u=P16), 1),
]


@pytest.mark.parametrize("args,status", FORWARD)
def test_forward_refusals(args, status):
    d = dict(act=1, x=P16, dt=hb.HYB_BF16, m=200, ldx=256, h=P16, ldh=128, g=P16, ldg=128, u=3 * P16, ldu=128, ws=P16,
             nbytes=1 << 40)
    d.update(args)
    st = gated.lib().hyb_gated(ctypes.byref(_packed_pair()), d["act"], d["x"], d["dt"], d["m"], d["ldx"], d["h"],
                               d["ldh"], d["g"], d["ldg"], d["u"], d["ldu"], d["ws"], d["nbytes"], None)
    assert _status(st) == status


@pytest.mark.parametrize("args,status", [
    (dict(act=9), 1), (dict(dt=hb.HYB_F32), 3), (dict(x=P16 + 1), 1), (dict(ldx=255), 1), (dict(h=None), 1),
    (dict(ldh=7), 1), (dict(g=P16, u=P16), 4), (dict(g=P16), 1), (dict(k=4, m=40, ws=None), 1), (dict(k=4, m=40, nbytes=5), 1),
])
def test_forward_4bit_refusals(args, status):
    d = dict(act=1, x=P16, dt=hb.HYB_BF16, m=2, k=256, ldx=256, h=P16, ldh=8, g=None, u=None, ws=P16, nbytes=1 << 40)
    d.update(args)
    st = gated.lib().hyb_gated(ctypes.byref(_q4_pair(k=d["k"])), d["act"], d["x"], d["dt"], d["m"], d["ldx"], d["h"], d["ldh"],
                               d["g"], 8, d["u"], 8, d["ws"], d["nbytes"], None)
    assert _status(st) == status


@pytest.mark.parametrize("args,status", [
    (dict(act=0), 1), (dict(dt=hb.HYB_F16), 3), (dict(m=-1), 2), (dict(x=P16 + 8), 1), (dict(ldx=257), 1),
    (dict(g=None), 1), (dict(u=None), 1), (dict(dh=None), 1), (dict(dh=P16 + 1), 1), (dict(lddh=100), 1),
    (dict(dx=P16 + 1), 1), (dict(lddx=200), 1), (dict(dwg=None), 1), (dict(dwu=None), 1), (dict(dwu=P16 + 1), 1),
    (dict(lddw=200), 1), (dict(ws=None), 1), (dict(nbytes=64), 1), (dict(dwu=P16), 1),
])
def test_backward_refusals(args, status):
    d = dict(act=1, x=P16, dt=hb.HYB_BF16, m=20, ldx=256, g=P16, u=P16, dh=P16, lddh=128, dx=P16, lddx=256, dwg=P16,
             dwu=3 * P16, lddw=256, ws=P16, nbytes=1 << 40)
    d.update(args)
    st = gated.lib().hyb_gated_backward(ctypes.byref(_packed_pair()), d["act"], d["x"], d["dt"], d["m"], d["ldx"],
                                        d["g"], 128, d["u"], 128, d["dh"], d["lddh"], d["dx"], d["lddx"], d["dwg"],
                                        d["lddw"], d["dwu"], d["lddw"], d["ws"], d["nbytes"], None)
    assert _status(st) == status


def test_4bit_weights_have_no_gradients():
    n = ctypes.c_size_t(0)
    L, w = gated.lib(), ctypes.byref(_q4_pair())
    assert _status(L.hyb_gated_workspace_size(w, 2, gated.DX, ctypes.byref(n))) == 4
    assert _status(L.hyb_gated_backward(w, 1, P16, hb.HYB_BF16, 2, 256, P16, 8, P16, 8, P16, 8, P16, 256, None, 0, None, 0,
                                        P16, 1 << 30, None)) == 4


def test_workspace_sizes():
    n = ctypes.c_size_t(0)
    L, w = gated.lib(), ctypes.byref(_packed_pair())

    def need(m, what, pair=w):
        assert L.hyb_gated_workspace_size(pair, m, what, ctypes.byref(n)) == 0
        return n.value
    assert need(0, 0) == need(0, 3) == 0
    assert _status(L.hyb_gated_workspace_size(w, -1, 0, ctypes.byref(n))) == 2
    assert _status(L.hyb_gated_workspace_size(w, 1, 4, ctypes.byref(n))) == 1
    assert _status(L.hyb_gated_workspace_size(w, 1, 0, None)) == 1
    dz = 2 * 208 * 128 * 2                                     # dG and dU of 200 tokens
    assert need(200, gated.DX) >= dz and need(200, gated.DW) >= dz
    assert need(200, gated.DX | gated.DW) >= max(need(200, gated.DX), need(200, gated.DW))
    four, narrow = ctypes.byref(_q4_pair()), ctypes.byref(_q4_pair(k=4))
    assert need(1, 0, four) == need(4, 0, four) == 0 and need(40, 0, narrow) >= 48 * 64 * 2


def test_empty_calls_do_nothing():
    L, w = gated.lib(), ctypes.byref(_packed_pair())
    assert L.hyb_gated(w, 1, None, hb.HYB_BF16, 0, 256, None, 128, None, 0, None, 0, None, 0, None) == 0
    assert L.hyb_gated_backward(w, 1, None, hb.HYB_BF16, 0, 256, None, 0, None, 0, None, 0, P16, 256, None, 0, None, 0,
                                None, 0, None) == 0
    assert L.hyb_gated_backward(w, 1, None, hb.HYB_BF16, 5, 256, None, 0, None, 0, None, 0, None, 0, None, 0, None, 0, None,
                                0, None) == 0
    assert L.hyb_gated(ctypes.byref(_q4_pair(n=0)), 1, None, hb.HYB_BF16, 3, 256, None, 0, None, 0, None, 0, None, 0,
                       None) == 0


def _fake(n, k, dtype="bf16"):
    L, tidx = hb.plan(n, k, 64, 64, dtype, "idx2", np.zeros(n // 64 * (k // 64)))
    return hb.allocate(L, tidx, "cpu", dtype, "idx2")


def _fake4(n, k):
    nc, ns = q4.sizes(n, k)
    return q4.Q4Matrix((n, k), torch.bfloat16, torch.empty(nc, dtype=torch.uint8), torch.empty(ns, dtype=torch.uint8))


def test_binding_refusals():
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    P, Q = _fake(64, 128), _fake4(64, 128)
    y, f = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, 64)
    for call, err in [
        (lambda: gated.forward(P, Q, x), TypeError), (lambda: gated.forward(x, x, x), TypeError),
        (lambda: gated.forward(P, _fake(128, 128), x), ValueError), (lambda: gated.forward(Q, _fake4(32, 128), x), ValueError),
        (lambda: gated.forward(P, _fake(64, 128, "f16"), x), TypeError),
        (lambda: gated.forward(P, P, x, act="relu"), ValueError), (lambda: gated.forward(P, P, x.half()), TypeError),
        (lambda: gated.forward(P, P, x[:, :64]), ValueError), (lambda: gated.forward(Q, Q, x.float()), TypeError),
        (lambda: gated.forward(Q, Q, x, save=True), TypeError), (lambda: gated.forward(P, P, x, out=x), ValueError),
        (lambda: gated.forward(P, P, x, out=y.float()), TypeError), (lambda: gated.forward(P, P, x), ValueError),
        (lambda: gated.backward(Q, Q, x, f, f, y), TypeError), (lambda: gated.backward(P, P, x, f, f, x), ValueError),
        (lambda: gated.backward(P, P, x, f, y, y), TypeError),
        (lambda: gated.backward(P, P, x, f, f, y, dw_gate=torch.zeros(64, 128, dtype=torch.bfloat16)), ValueError),
        (lambda: gated.backward(P, P, x, f, f, y, dx=y), ValueError),
        (lambda: gated.backward(P, P, x, f, f, y), ValueError),              # not on a GPU
    ]:
        with pytest.raises(err):
            call()
