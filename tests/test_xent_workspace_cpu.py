"""Workspace of the cross entropy over heads without sparse tiles, which are
multiplied where they lie: what the operands and sums need, not a copy of the
head.

Bounds, with m16 = m rounded up to 16: x in panels m16 k 2; loss: softmax sums 8
m16 per 256 entries; gradients: dz m16 n 2 (at most 256 MiB), at most 32 parts
of dX (m k 4), one tile row b1 k 2; up to 64 tokens the fp32 logits m n 4.  Each
buffer is rounded up to 256 bytes."""
import ctypes

import numpy as np
import pytest

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import xent

MIB = 1 << 20


def size(n, k, b, m, what):
    L, _ = hb.plan(n, k, b, b, "bf16", "idx2", np.zeros((n // b) * (k // b), np.uint8))
    P = hb.HybPacked(None, None, None, None)
    head = xent.HybHead(ctypes.pointer(L), ctypes.pointer(P), None, n, k)
    nbytes = ctypes.c_size_t(0)
    hb.check(xent.lib().hyb_xent_workspace_size(ctypes.byref(head), m, what, ctypes.byref(nbytes)), "size")
    return nbytes.value


@pytest.mark.parametrize("b", [64, 128, 256])
@pytest.mark.parametrize("n,k", [(128256, 4096), (128256, 8192), (32768, 4096), (152064, 5120)])
@pytest.mark.parametrize("m", [1, 16, 64, 65, 100, 2048, 20000])
def test_dense_heads_are_not_copied(m, n, k, b):
    n = n // b * b
    m16 = -(-m // 16) * 16
    logits = m * n * 4 if m <= 64 else 0
    assert size(n, k, b, m, 0) <= m16 * k * 2 + logits + 8 * m16 * -(-n // 256) + 4 * m16 + 6 * 256
    dz = min(m16 * (n + 255) * 2, max(256 * MIB, m16 * 512))
    for what in (xent.DX, xent.DW, xent.DX | xent.DW):
        assert size(n, k, b, m, what) <= m16 * k * 2 + logits + dz + 32 * m * k * 4 + b * k * 2 + 7 * 256


def test_a_hundred_tokens_over_a_large_head():
    assert size(128256, 4096, 128, 100, 0) < 2 * MIB
    assert size(128256, 4096, 128, 2048, 0) < 25 * MIB
    assert size(128256, 4096, 128, 16, xent.DX) < 24 * MIB
