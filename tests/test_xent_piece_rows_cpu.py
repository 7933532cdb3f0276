"""hyb_xent_piece_rows: its refusals, and how heads are cut (256 compute units, or
the device's)."""
import ctypes

import numpy as np
import pytest

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import f8, xent

P16 = 1 << 20  # any 16-byte aligned non-null address: never followed


def packed(n, k=64, sparse=False):
    L, _ = hb.plan(n, k, 64, 64, "bf16", "idx2", np.arange((n // 64) * (k // 64)) % 2 * int(sparse))
    return xent.HybHead(ctypes.pointer(L), ctypes.pointer(hb.HybPacked(None, None, None, None)), None, n, k)


def codes(n, k=64):
    return xent.HybHead(None, None, ctypes.pointer(f8.HybF8(P16, P16)), n, k)


def call(head, m, what, rows):
    return xent.lib().hyb_xent_piece_rows(head, m, what, rows)


def rows(head, m, what):
    out = ctypes.c_int64(0)
    hb.check(call(ctypes.byref(head), m, what, ctypes.byref(out)), "rows")
    return out.value


@pytest.mark.parametrize("head", [lambda n: packed(n), lambda n: packed(n, sparse=True), codes])
def test_pieces(head):
    for what in (xent.DX, xent.DX | xent.DW) if head is not codes else (xent.DX,):
        assert rows(head(66048), 1000, what) == 32768           # 64 MiB of dz
        assert rows(head(66048), 20000, what) == 6656           # 256 MiB of dz
        assert rows(head(270080), 100, what) < 270080           # few tokens take more
        assert rows(head(600064), 16, what) < 600064
        assert rows(head(9024), 16, what) == 9024
    assert rows(head(600064), 16, 0) == 600064                  # logits through the library's product


def test_pieces_of_the_loss():
    assert rows(packed(66048), 1000, 0) == 66048 and rows(codes(66048), 1000, 0) == 66048   # multiplied where it lies
    assert rows(packed(66048, sparse=True), 200, 0) == 32768
    assert rows(packed(66048, sparse=True), 600, 0) < 66048


@pytest.mark.parametrize("args,status", [
    (dict(m=0), 2), (dict(m=-1), 2), (dict(m=(1 << 22) + 1), 2), (dict(what=4), 1), (dict(what=-1), 1), (dict(head=None), 1),
    (dict(rows=None), 1), (dict(head=ctypes.byref(xent.HybHead())), 1), (dict(head=ctypes.byref(codes(300)), what=2), 4),
])
def test_refusals(args, status):
    d = dict(head=ctypes.byref(packed(256)), m=4, what=1, rows=ctypes.byref(ctypes.c_int64(0)))
    d.update(args)
    with pytest.raises(hb.HybError) as e:
        hb.check(call(d["head"], d["m"], d["what"], d["rows"]), "call")
    assert e.value.status == status
