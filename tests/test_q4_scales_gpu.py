"""fp16 products over 4-bit weights at the ends of what hyb_q4.h promises: rows of
any scale beside groups of zeros."""
import pytest
import torch

from matmul_pack_b1_amd import gated, q4

pytestmark = pytest.mark.gpu

GRID = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def rows_of_every_scale(k, live):
    """251 rows, row i of values code * 2^(i - 125) in columns 0 .. live - 1 (float64;
    a largest of 6 * 2^e has the scale 2^e), and the weight in 4 bits."""
    w = torch.zeros(251, k, dtype=torch.float64)
    for i in range(251):
        w[i, :live] = GRID[(torch.arange(live) + i) % 7] * 2.0 ** (i - 125) * (1 - 2 * (torch.arange(live) % 2))
        w[i, 0] = 6 * 2.0 ** (i - 125)
    Q = q4.pack(w.float().cuda())
    assert torch.equal(q4.unpack(Q, out_dtype=torch.float32).double().cpu(), w)
    return Q, w


# (columns, columns that are not zero, tokens): the kernel of few tokens, the one
# that shares activations (one to several parts), the tiles (rows of 7 columns)
WAYS = [(320, 32, 1), (320, 32, 2), (320, 32, 4), (320, 32, 9), (320, 20, 40), (5000, 32, 20), (33, 32, 70), (40, 7, 6),
        (7, 7, 5), (7, 7, 140)]


@pytest.mark.parametrize("k,live,m", WAYS)
def test_rows_of_any_scale_beside_zeros(k, live, m):
    """Integers of up to 5 bits times codes: every sum is exact, down to where fp32
    itself ends (a half step of its smallest number, 2^-150)."""
    Q, w = rows_of_every_scale(k, live)
    x = torch.randint(-15, 16, (m, k), generator=torch.Generator().manual_seed(k + m)).double() / 1024
    ref = x @ w.t()
    y = q4.gemm(Q, x.half().cuda()).double().cpu()
    bad = (~((y - ref).abs() <= 2.0 ** -150)).nonzero()
    assert len(bad) == 0, (len(bad), bad[:4].tolist(), sorted({int(c) for c in bad[:, 1]})[:8])


@pytest.mark.parametrize("k,live,m", WAYS)
def test_gated_rows_of_any_scale_beside_zeros(k, live, m):
    """H = silu(G) U, one weight's rows as above, the other's 1 in a column: nothing is
    NaN, and what fp16 holds is right: half a step, and (|g| + 4) * 2^-22 for the
    exponential, the reciprocal and two products in fp32."""
    Q, w = rows_of_every_scale(k, live)
    ones = torch.zeros(251, k, dtype=torch.float64)
    ones[:, 0] = 1.0
    x = torch.randint(-15, 16, (m, k), generator=torch.Generator().manual_seed(k + m)).double() / 1024
    u = x @ w.t()
    for gate, up in ((ones, w), (w, ones)):
        A, B = (Q if t is w else q4.pack(ones.float().cuda()) for t in (gate, up))
        g, u = x @ gate.t(), x @ up.t()
        ref = g * torch.sigmoid(g) * u
        h = gated.forward(A, B, x.half().cuda()).double().cpu()
        assert not bool(h.isnan().any())
        fits = (ref.abs() < 60000) & (g.abs() < 8)
        assert bool(((h - ref).abs() <= (2.0 ** -11 + 2.0 ** -17) * ref.abs() + 2.0 ** -25)[fits].all())
