"""fp16 products over 4-bit weights at the ends of what hyb_q4.h promises: rows of
any scale beside groups of zeros, and groups far below their row's largest."""
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


# As above, with the columns of the two groups.
FAR = [(64, 1), (64, 3), (64, 4), (64, 16), (320, 40), (5000, 30), (64, 70), (64, 64)]


@pytest.mark.parametrize("k,m", FAR)
@pytest.mark.parametrize("below", [26, 30, 35, 36])
def test_groups_far_below_their_row(k, m, below):
    """Scales of 2^-36 of the row's largest and above are exact: one activation a
    token, in the small group."""
    w = torch.zeros(70, k, dtype=torch.float64)
    for r in range(70):
        sign = 1 - 2 * (torch.arange(32) % 2)
        w[r, :32] = 6.0 * 2.0 ** (r - 20)
        w[r, 32:64] = GRID[(torch.arange(32) + r) % 7] * sign * 2.0 ** (r - 20 - below)
        w[r, 32 + (r + 3) % 32] = 6.0 * 2.0 ** (r - 20 - below)
    Q = q4.pack(w.float().cuda())
    assert torch.equal(q4.unpack(Q, out_dtype=torch.float32).double().cpu(), w)
    x = torch.zeros(m, k, dtype=torch.float64)
    x[torch.arange(m), 32 + torch.arange(m) % 32] = 1.0 + torch.arange(m).double() / 1024
    y = q4.gemm(Q, x.half().cuda()).double().cpu()
    assert torch.equal(y, x @ w.t())


@pytest.mark.parametrize("m", [333, 901])
@pytest.mark.parametrize("below", [26, 35, 36])
def test_groups_far_below_their_row_in_tiles(m, below):
    """The same in the LDS-fed tiles (128 and 256 tokens; gated whole and cut)."""
    n, k = 12003, 515
    w = torch.zeros(n, k, dtype=torch.float64, device="cuda")
    w[:, :32] = 6.0
    w[:, 480:512] = GRID.cuda()[(torch.arange(n, device="cuda")[:, None] + torch.arange(32, device="cuda")) % 7] * 2.0 ** -below
    w[torch.arange(n), 480 + torch.arange(n) % 32] = 6.0 * 2.0 ** -below
    Q = q4.pack(w.float())
    x = torch.zeros(m, k, dtype=torch.float64, device="cuda")
    x[torch.arange(m), 480 + torch.arange(m) % 32] = 1.0 + torch.arange(m, device="cuda").double() / 1024
    ref = x @ w.t()
    assert torch.equal(q4.gemm(Q, x.half()).double(), ref)
    # the gated tiles: silu(32) is 32 in fp32
    w2 = torch.zeros_like(w)
    w2[:, 512] = 2.0
    x[:, 512] = 16.0
    big = 2.0 ** 31
    x[:, 480:512] *= 2.0 ** 10
    up = w * big / 2.0 ** 10
    h = gated.forward(q4.pack(w2.float()), q4.pack(up.float()), x.half()).double()
    want = (32.0 * (x @ up.t())).half().double()
    assert torch.equal(h, want)
