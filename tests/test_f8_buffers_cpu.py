"""F8Matrix buffers that no kernel may be given: on two devices, not bytes, not
contiguous.  Refused by every call that takes one, before the library is."""
import pytest
import torch

from matmul_pack_b1_amd import f8, xent


def matrix(kind=f8.WEIGHT, rows=40, k=300):
    nc, ns = f8.sizes(rows, k)
    return f8.F8Matrix(kind, (rows, k), torch.bfloat16, torch.empty(nc, dtype=torch.uint8),
                       torch.empty(ns, dtype=torch.uint8))


def spoiled(how, kind=f8.WEIGHT):
    Q = matrix(kind)
    if how == "device":
        Q.scales = Q.scales.to("meta")
    elif how == "type":
        Q.codes = torch.empty(Q.codes.numel(), dtype=torch.int32)
    elif how == "stride":
        Q.codes = torch.empty(2 * Q.codes.numel(), dtype=torch.uint8)[::2]
    else:
        Q.scales = torch.empty(2 * Q.scales.numel(), dtype=torch.uint8)[::2]
    return Q


@pytest.mark.parametrize("how,err,text", [("device", ValueError, "scales are on meta"), ("type", TypeError, "int32"),
                                          ("stride", ValueError, "contiguous"), ("stride of scales", ValueError, "contiguous")])
def test_refused(how, err, text):
    x, t = torch.zeros(4, 300, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: f8.gemm(spoiled(how), x), lambda: f8.gemm(matrix(), spoiled(how, f8.ROWS)),
                 lambda: f8.unpack(spoiled(how)), lambda: f8.pack(torch.zeros(40, 300), out=spoiled(how)),
                 lambda: xent.loss(spoiled(how), x, t), lambda: xent.workspace_bytes(spoiled(how), 4)):
        with pytest.raises(err, match=text):
            call()


def test_whole_buffers_pass():
    f8._check_matrix(matrix(), f8.WEIGHT, "Q")
    with pytest.raises(ValueError, match="on a GPU"):
        f8.gemm(matrix(), torch.zeros(4, 300, dtype=torch.bfloat16))
