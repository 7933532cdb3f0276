"""Every tile and way of cutting of the gated projection over packed weights and of
its gradients (route_shapes.py) against float64.

Forward: G and U are fp32 sums of exact products, off by at most k * 2^-23 * S, S =
sum |x w|; act has a slope of at most 1.2 and is itself off by (|g|^3 + |g| + 8) *
2^-23 * |g|; H is rounded to 16 bits.  Backward, from the call's own G and U: dG and dU
are off by the slope's error (one power of g more) and half a step (fp16 holds them
scaled, off by 2^-37 of the largest at least), sums by 2^-23 of the absolute sum a
term, and each output is rounded by half a step."""
import numpy as np
import pytest
import torch

import route_shapes as rs
from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
TYPES = [torch.bfloat16, torch.float16]


def normal(seed, rows, cols, dtype, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(dtype)


def weight(seed, n, k, dtype):
    """A weight with half of its tiles sparse, and what its streams stand for (the
    read-back has tests of its own)."""
    tiles = (np.random.default_rng(seed).random((n // 64, k // 64)) < 0.5).astype(np.uint8)
    P = hb.pack(normal(seed, n, k, dtype, k ** -0.5), tiles, 64, 64, "idx2")
    return P, hb.unpack(P).double()


def close(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = (~(err <= tol)).nonzero()
    assert len(bad) == 0, (len(bad), bad[:4].tolist(), float((err - tol).max()))


def act_error(g):
    return (g ** 3 + g + 8.0) * 2.0 ** -23 * g


def check_forward(x, wg, wu, out, dtype):
    xd, k = x.double(), x.shape[1]
    refs = [xd @ w.t() for w in (wg, wu)]
    errs = [k * 2.0 ** -23 * (xd.abs() @ w.abs().t()) for w in (wg, wu)]
    h, gu = (out[0], out[1:]) if isinstance(out, tuple) else (out, ())
    for got, ref, err in zip(gu, refs, errs):
        close(got, ref, err)
    (g, u), (eg, eu) = refs, errs
    a = g * torch.sigmoid(g)
    ea = 1.2 * eg + act_error(g.abs() + eg)
    tol = (a.abs() + ea) * eu + ea * u.abs()
    close(h, a * u, tol + HALF[dtype] * ((a * u).abs() + tol) + LEAST[dtype])


@pytest.mark.parametrize("case", list(rs.GATED_FORWARD), ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_forward(case, dtype):
    n, k, m = rs.GATED_FORWARD[case]
    (G, wg), (U, wu) = weight(n + k, n, k, dtype), weight(n + k + 1, n, k, dtype)
    x = normal(m, m, k, dtype)
    kept = gated.forward(G, U, x, save=True)
    check_forward(x, wg, wu, kept, dtype)
    assert torch.equal(gated.forward(G, U, x), kept[0])


@pytest.mark.parametrize("case", list(rs.GATED_BACKWARD), ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward(case, dtype):
    n, k, m = rs.GATED_BACKWARD[case]
    (G, wg), (U, wu) = weight(n + k, n, k, dtype), weight(n + k + 1, n, k, dtype)
    x, dh = normal(m, m, k, dtype), normal(m + 1, m, n, dtype, 0.1)
    _, g, u = gated.forward(G, U, x, save=True)
    dx, dwg, dwu = gated.backward(G, U, x, g, u, dh, need_dw=True)
    gd, ud, dd, xd = g.double(), u.double(), dh.double(), x.double()
    s = torch.sigmoid(gd)
    a, slope = gd * s, s * (1.0 + gd * (1.0 - s))
    dg, du = dd * ud * slope, dd * a
    es = (gd.abs() ** 3 + gd.abs() + 8.0) * 2.0 ** -22 * (1.0 + gd.abs())
    eg = (dd * ud).abs() * (es + 2.0 ** -22 * slope.abs())
    eu = dd.abs() * (act_error(gd.abs()) + 2.0 ** -23 * a.abs())
    least = max(float(dg.abs().max()), float(du.abs().max())) * 2.0 ** -37 if dtype == torch.float16 else 0.0
    eg = eg + HALF[dtype] * (dg.abs() + eg) + least
    eu = eu + HALF[dtype] * (du.abs() + eu) + least
    ag, au = dg.abs() + eg, du.abs() + eu

    def rounded(ref, tol):
        return tol + HALF[dtype] * (ref.abs() + tol) + LEAST[dtype]

    ref = dg @ wg + du @ wu
    sums = ag @ wg.abs() + au @ wu.abs()
    close(dx, ref, rounded(ref, eg @ wg.abs() + eu @ wu.abs() + 2 * n * 2.0 ** -23 * sums))
    for got, d, e, ad in ((dwg, dg, eg, ag), (dwu, du, eu, au)):
        ref = d.t() @ xd
        close(got, ref, rounded(ref, e.t() @ xd.abs() + m * 2.0 ** -23 * (ad.t() @ xd.abs())))
    # one gradient alone, and both again: the same bits
    assert torch.equal(gated.backward(G, U, x, g, u, dh)[0], dx)
    alone = gated.backward(G, U, x, g, u, dh, need_dx=False, need_dw=True)
    assert torch.equal(alone[1], dwg) and torch.equal(alone[2], dwu)
