"""The smallest of the fp16 gradients that the gated projection's backward pass
holds scaled (hyb_gated.h)."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [2, 70, 300])
@pytest.mark.parametrize("top", [1.0, 2.0 - 2.0 ** -10])
@pytest.mark.parametrize("below", [20, 27, 28])
def test_smallest_fp16_gradients(below, top, m):
    """dU of 2^-28 of the largest and above keep their eleven bits: silu(32) is 32 in
    fp32, u = 0 leaves dG out, and W_u is the identity, so that dX and dW_u hold dU."""
    n = k = 128
    eye = torch.eye(n, dtype=torch.float16, device="cuda")
    P = hb.pack(eye, np.zeros((2, 2), dtype=np.uint8), 64, 64, "idx2")
    g, u = torch.full((m, n), 32.0, device="cuda"), torch.zeros(m, n, device="cuda")
    bits = 1.0 + (torch.arange(n, dtype=torch.float64) * 8 + 1) / 1024      # odd in the last place
    bits[0] = 1.0
    # dU = 32 dh: the largest top * 2^15 in one token, the others' 2^(15 - below)
    dh = (bits * 2.0 ** (10 - below)).repeat(m, 1)
    dh[0] = 0.0
    dh[0, 5] = top * 2.0 ** 10
    if below > 24:       # (dh itself has to be normal in fp16)
        dh[0, 5] *= 2.0 ** 5
        dh[1:] *= 2.0 ** 5
    small = dh[m - 1] * 32.0
    dh = dh.half().cuda()
    assert torch.equal(dh[m - 1].double().cpu() * 32.0, small)
    x = torch.zeros(m, k, dtype=torch.float16, device="cuda")
    x[m - 1, 77] = 64.0
    dx, dwg, dwu = gated.backward(P, P, x, g, u, dh, need_dw=True)
    assert torch.equal(dwu[:, 77].double().cpu(), 64.0 * small)
    assert not dwg.any() and not dwu[:, :77].any() and not dwu[:, 78:].any()
    # (dX is rounded to fp16, whose normal numbers end at 2^-14)
    assert torch.equal(dx[m - 1].cpu(), small.half())


@pytest.mark.parametrize("m", [2, 300])
@pytest.mark.parametrize("size", [2.0 ** -125, 2.0 ** -80, 2.0 ** 80, 2.0 ** 112])
def test_largest_of_any_size(size, m):
    """A largest dG anywhere in fp32: finite, so that it adds nothing where it meets
    zeros, and right where an output holds it (infinite beyond fp16, 0 below it)."""
    n = k = 128
    P = hb.pack(torch.eye(n, dtype=torch.float16, device="cuda"), np.zeros((2, 2), dtype=np.uint8), 64, 64, "idx2")
    g, u = torch.full((m, n), 32.0, device="cuda"), torch.zeros(m, n, device="cuda")
    dh = torch.zeros(m, n, dtype=torch.float16, device="cuda")
    dh[0], u[0] = 2.0 ** 15, size / 2.0 ** 2     # dG = 2^13 size, dU = 2^20
    dh[0, 1:] = 0.0
    x = torch.zeros(m, k, dtype=torch.float16, device="cuda")
    x[0, 3] = 2.0 ** -10
    dx, dwg, dwu = gated.backward(P, P, x, g, u, dh, need_dw=True)
    dg = 2.0 ** 13 * size
    assert not dwg[1:].any() and not dwg[0, :3].any() and not dwg[0, 4:].any()
    assert float(dwg[0, 3]) == float(torch.tensor(dg * 2.0 ** -10, dtype=torch.float64).half())
    assert not dx[1:].any() and not dx[0, 1:].any() and float(dx[0, 0]) == float("inf")
    if size < 1:
        assert float(dwu[0, 3]) == 2.0 ** 10
