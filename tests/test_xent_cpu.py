"""Cross entropy over a vocabulary projection without a GPU: the C ABI's
refusals and workspace sizes (include/hyb_xent.h), the binding's checks, and
the gradient formula against differences."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import f8, xent
from oracle import xent_oracle as xo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P16 = 1 << 20  # any 16-byte aligned non-null address: never followed


def test_exports_match_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hyb_xent.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(hyb_[a-z0-9_]+)\s*\(", text))
    assert names == set(xent.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", hb.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (hyb_\w+)", out))


def packed_head(n=256, k=128, dtype="bf16", streams=True, b1=64, b2=64):
    L, _ = hb.plan(n, k, b1, b2, dtype, "idx2", np.arange((n // b1) * (k // b2)) % 2)
    P = hb.HybPacked(P16, P16, P16, P16) if streams else hb.HybPacked(None, None, None, None)
    return xent.HybHead(ctypes.pointer(L), ctypes.pointer(P), None, n, k)


def f8_head(n=300, k=200, codes=P16):
    return xent.HybHead(None, None, ctypes.pointer(f8.HybF8(codes, P16)), n, k)


def _status(st):
    with pytest.raises(hb.HybError) as e:
        hb.check(st, "call")
    return e.value.status


def size(head, m, what):
    n = ctypes.c_size_t(0)
    hb.check(xent.lib().hyb_xent_workspace_size(ctypes.byref(head), m, what, ctypes.byref(n)), "size")
    return n.value


@pytest.mark.parametrize("head", [packed_head, f8_head])
def test_workspace_sizes(head):
    assert size(head(), 0, 0) == 0
    for what in (0, 1) if head is f8_head else (0, 1, 2, 3):
        small = [size(head(), m, what) for m in (1, 64, 65, 2000, 100000)]
        assert all(a <= b for a, b in zip(small[2:], small[3:])) and all(s > 0 and s % 256 == 0 for s in small)
    # the loss alone never holds logits of many tokens: 4096 x 128256 fp32 are 2.1 GB
    assert size(packed_head(128256, 4096, b1=64, b2=128), 4096, 0) < 400 << 20


FWD = dict(head=packed_head, n_vocab=250, x=P16, dt=hb.HYB_BF16, m=4, ldx=128, target=P16, loss=P16, lse=P16, ws=P16,
           nbytes=1 << 40)


def forward(d):
    head = d["head"]()
    return xent.lib().hyb_xent(ctypes.byref(head), d["n_vocab"], d["x"], d["dt"], d["m"], d["ldx"], d["target"], -100,
                               d["loss"], d["lse"], d["ws"], d["nbytes"], None)


def back(d):
    head = d["head"]()
    return xent.lib().hyb_xent_backward(ctypes.byref(head), d["n_vocab"], d["x"], d["dt"], d["m"], d["ldx"],
                                        d["target"], -100, d["lse"], d["loss"], d["dx"], d["lddx"], d["dw"], d["lddw"],
                                        d["ws"], d["nbytes"], None)


BOTH_REFUSALS = [
    (dict(n_vocab=0), 2), (dict(n_vocab=257), 2), (dict(m=-1), 2), (dict(m=(1 << 22) + 1), 2), (dict(dt=hb.HYB_F32), 3),
    (dict(dt=hb.HYB_F16), 3), (dict(x=None), 1), (dict(x=P16 + 8), 1), (dict(ldx=120), 1), (dict(ldx=132), 1),
    (dict(ldx=1 << 22), 4), (dict(target=None), 1), (dict(target=P16 + 4), 1), (dict(nbytes=255), 1), (dict(ws=None), 1),
    (dict(ws=P16 + 8), 1), (dict(loss=None), 1), (dict(lse=None), 1), (dict(lse=P16 + 2), 1),
    (dict(head=lambda: packed_head(streams=False)), 1), (dict(head=lambda: f8_head(codes=None)), 1),
    (dict(head=lambda: f8_head(codes=P16 + 4)), 1), (dict(head=lambda: f8_head(n=0)), 2),
    (dict(head=lambda: f8_head(k=0)), 2), (dict(head=lambda: f8_head(k=(1 << 21) + 1)), 2),
    (dict(head=lambda: f8_head(n=(1 << 27))), 2), (dict(head=lambda: xent.HybHead()), 1),
    (dict(head=lambda: f8_head(n=(1 << 27) - 16, k=128), m=1 << 20), 4),
    (dict(head=lambda: packed_head(b1=80, n=240, k=128), n_vocab=240), 4),
]


@pytest.mark.parametrize("args,status", BOTH_REFUSALS)
def test_refusals(args, status):
    d = dict(FWD, **args)
    assert _status(forward(d)) == status
    d.update(dx=P16, lddx=128 if "head" not in args else 1 << 21, dw=None, lddw=0)
    if status != 1 or "loss" not in args:
        assert _status(back(d)) == status


@pytest.mark.parametrize("args,status", [
    (dict(dx=P16 + 1), 1), (dict(lddx=127), 1), (dict(dw=P16 + 1), 1), (dict(lddw=100), 1),
    (dict(lddw=(1 << 31) + 1), 4), (dict(lddx=(1 << 31) + 1), 4), (dict(head=f8_head, ldx=200, lddx=200, lddw=200), 4),
])
def test_backward_refusals(args, status):
    d = dict(FWD, dx=P16, lddx=128, dw=P16, lddw=128)
    d.update(args)
    assert _status(back(d)) == status


def test_both_forms_at_once_is_refused():
    both = packed_head()
    both.f8 = ctypes.pointer(f8.HybF8(P16, P16))
    assert _status(forward(dict(FWD, head=lambda: both))) == 1
    n = ctypes.c_size_t(0)
    L = xent.lib()
    assert _status(L.hyb_xent_workspace_size(ctypes.byref(f8_head()), 4, 2, ctypes.byref(n))) == 4
    assert _status(L.hyb_xent_workspace_size(ctypes.byref(f8_head()), 4, 4, ctypes.byref(n))) == 1
    assert _status(L.hyb_xent_workspace_size(ctypes.byref(f8_head()), -1, 0, ctypes.byref(n))) == 2
    assert _status(L.hyb_xent_workspace_size(ctypes.byref(f8_head()), 4, 0, None)) == 1
    assert _status(L.hyb_xent_workspace_size(None, 4, 0, ctypes.byref(n))) == 1


def test_empty_calls_do_nothing():
    assert forward(dict(FWD, m=0, x=None, target=None, loss=None, lse=None, ws=None, nbytes=0)) == 0
    d = dict(FWD, dx=P16, lddx=128, dw=None, lddw=0)
    assert back(dict(d, m=0)) == 0
    assert back(dict(d, dx=None)) == 0


def test_binding_refusals():
    nc, ns = f8.sizes(300, 200)
    Q = f8.F8Matrix(f8.WEIGHT, (300, 200), torch.bfloat16, torch.empty(nc, dtype=torch.uint8),
                    torch.empty(ns, dtype=torch.uint8))
    x, t = torch.zeros(4, 200, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    for call, err in [
        (lambda: xent.loss(x, x, t), TypeError), (lambda: xent.loss(Q, x.float(), t), TypeError),
        (lambda: xent.loss(Q, x[:, :100], t), ValueError), (lambda: xent.loss(Q, x, t.int()), TypeError),
        (lambda: xent.loss(Q, x, t[:3]), ValueError), (lambda: xent.loss(Q, x, t[:, None]), ValueError),
        (lambda: xent.loss(Q, x, torch.zeros(8, dtype=torch.int64)[::2]), ValueError),
        (lambda: xent.loss(Q, x.t(), t), ValueError), (lambda: xent.loss(Q, x, t), ValueError),   # not on a GPU
    ]:
        with pytest.raises(err):
            call()


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((5, 7)), rng.standard_normal((11, 7))
    target = np.array([0, 8, -100, 3, 8])
    grad = rng.standard_normal(5)
    _, _, dx, dw = xo.cross_entropy(x, w, target, 9, grad=grad)
    total = lambda a, b: float((xo.cross_entropy(a, b, target, 9)[0] * grad).sum())
    for a, d, pick in ((x, dx, 0), (w, dw, 1)):
        for idx in np.ndindex(a.shape):
            lo, hi = a.copy(), a.copy()
            lo[idx] -= 1e-5
            hi[idx] += 1e-5
            diff = (total(hi, w) - total(lo, w) if pick == 0 else total(x, hi) - total(x, lo)) / 2e-5
            assert abs(diff - d[idx]) < 1e-8
    assert np.all(dx[2] == 0) and np.all(dw[9:] == 0)
