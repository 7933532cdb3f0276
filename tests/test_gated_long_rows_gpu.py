"""The gated projection and its gradients over rows of many columns (n k is what the
launches bound, not k alone).  X of -1, 0 and 1 and weights of small whole numbers make
G and U exact; H and the gradients are off by their roundings to 16 bits (2^-8 each)
and by the fp32 sums of the gradients (2^-23 of the absolute sum a term), the gradients'
own two factors by 2^-20."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [(1 << 18) + 64, 1 << 21])
@pytest.mark.parametrize("m", [1, 9, 40, 140])
def test_long_rows(k, m):
    n, gen = 64, torch.Generator("cuda").manual_seed(m)
    tiles = (np.arange(k // 64) % 2).astype(np.uint8)
    Ws = [hb.pack(torch.randint(-4, 5, (n, k), generator=gen, device="cuda").to(torch.bfloat16), tiles, 64, 64, "idx2")
          for _ in range(2)]
    wg, wu = (hb.unpack(W).float() for W in Ws)
    x = (torch.randint(0, 3, (m, k), generator=gen, device="cuda") - 1).to(torch.bfloat16)
    x[:, torch.rand(k, generator=gen, device="cuda") < 0.999] = 0
    h, g, u = gated.forward(*Ws, x, save=True)
    xf = x.float()
    assert torch.equal(g, xf @ wg.t()) and torch.equal(u, xf @ wu.t())
    gd, ud = g.double(), u.double()
    s = torch.sigmoid(gd)
    ref = gd * s * ud
    assert bool(((h.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 1e-9).all())
    dh = torch.randn(m, n, generator=gen, device="cuda").to(torch.bfloat16)
    dx, dwg, dwu = gated.backward(*Ws, x, g, u, dh, need_dw=True)
    # what the products are given: dG and dU of the slopes in float64, in bf16
    dg, du = dh.double() * ud * s * (1.0 + gd * (1.0 - s)), dh.double() * gd * s
    off = 2.0 ** -8 + 2.0 ** -16
    for got, d in ((dwg, dg), (dwu, du)):
        ref, most = d.t().float() @ xf, d.t().abs().float() @ xf.abs()
        assert bool(((got.float() - ref).abs() <= (2 * off + m * 2.0 ** -22) * most + 1e-6).all())
    ref = dg.float() @ wg + du.float() @ wu
    most = dg.abs().float() @ wg.abs() + du.abs().float() @ wu.abs()
    assert bool(((dx.float() - ref).abs() <= (2 * off + 2 * n * 2.0 ** -22) * most + 1e-6).all())
