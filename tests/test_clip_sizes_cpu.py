"""Sizing the workspace of a norm, whose tensors have no output (hyb_clip.h)."""
import ctypes

import pytest

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import clip


def need(*ts):
    n = ctypes.c_size_t(0)
    hb.check(clip.lib().hyb_clip_workspace_size(len(ts), (clip.HybTensor * len(ts))(*ts), ctypes.byref(n)), "size")
    return n.value


def tensor(rows, cols, lda, ldo):
    return clip.HybTensor(None, None, rows, cols, lda, ldo, hb.HYB_F32)


@pytest.mark.parametrize("ldo", [0, -5, 7, 1 << 62, -(1 << 63)])
def test_an_output_that_is_not_given_is_not_looked_at(ldo):
    assert need(tensor(3, 8, 9, ldo)) == need(tensor(3, 8, 9, 9)) == 24     # a chunk for each row apart
    assert need(tensor(4, 8, 8, ldo)) == need(tensor(4, 8, 8, 8)) == 8


def test_an_output_that_is_given_counts():
    assert need(tensor(4, 8, 8, 9)) == 32


@pytest.mark.parametrize("lda", [7, -1, (1 << 40) + 1])
def test_the_data_is_still_checked(lda):
    with pytest.raises(hb.HybError):
        need(tensor(4, 8, lda, 0))
