"""Every kernel, tile and way of cutting of the 4-bit products (route_shapes.py)
against products in float64 of the values read back (which have tests of their own
against the oracle).

A product's terms are exact, so its fp32 sum is off by at most k * 2^-23 * S, S =
sum |x w|, and a 16-bit output by half a step (2^-8, 2^-11) more.  The gated product:
act has a slope of at most 1.2, and is off by (|g|^3 + |g| + 8) * 2^-23 * |g| itself."""
import pytest
import torch

import route_shapes as rs
from matmul_pack_b1_amd import gated, q4

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
TYPES = [torch.bfloat16, torch.float16]


def normal(seed, rows, cols, dtype, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(dtype)


def weight(seed, n, k):
    Q = q4.pack(normal(seed, n, k, torch.bfloat16, k ** -0.5))
    return Q, q4.unpack(Q, out_dtype=torch.float32).double()


def close(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = (~(err <= tol)).nonzero()
    assert len(bad) == 0, (len(bad), bad[:4].tolist(), float((err - tol).max()))


def check(n, k, m, dtype, out):
    """x and y inside wider buffers, whose other elements stay out of the sums
    and as they were."""
    Q, w = weight(n + k, n, k)
    wide = torch.full((m + 1, k + 9), float("nan"), dtype=dtype, device="cuda")
    wide[:m, 3:k + 3] = normal(m, m, k, dtype)
    x = wide[:m, 3:k + 3]
    base = torch.full((m + 1, n + 7), 7.0, dtype=out, device="cuda")
    y = q4.gemm(Q, x, out=base[:m, 1:n + 1])
    xd = x.double()
    ref = xd @ w.t()
    close(y, ref, k * 2.0 ** -23 * (xd.abs() @ w.abs().t()) + HALF[out] * ref.abs() + LEAST[out])
    z = y.clone()
    y.fill_(7.0)
    assert bool((base == 7.0).all())
    assert torch.equal(z, q4.gemm(Q, x.contiguous(), out_dtype=out))   # and again the same


@pytest.mark.parametrize("case", [c for c in rs.Q4 if c[0] == 1], ids=str)
@pytest.mark.parametrize("dtype,wide", [(torch.bfloat16, False), (torch.float16, True)])
def test_product(case, dtype, wide):
    check(*rs.Q4[case], dtype, torch.float32 if wide else dtype)


@pytest.mark.parametrize("shape", rs.Q4_NARROW)
@pytest.mark.parametrize("dtype", TYPES)
def test_narrow_products(shape, dtype):
    check(*shape, dtype, torch.float32)
    check(*shape, dtype, dtype)


@pytest.mark.parametrize("case,shape", [(c, s) for c, s in rs.Q4.items() if c[0] == 2] +
                         [("narrow", s) for s in rs.Q4_NARROW], ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_gated(case, shape, dtype):
    n, k, m = shape
    (G, wg), (U, wu) = weight(n + k, n, k), weight(n + k + 1, n, k)
    x = normal(m, m, k, dtype)
    xd = x.double()
    g, u = xd @ wg.t(), xd @ wu.t()
    eg, eu = (k * 2.0 ** -23 * (xd.abs() @ w.abs().t()) for w in (wg, wu))
    a = g * torch.sigmoid(g)
    far = g.abs() + eg
    ea = 1.2 * eg + (far ** 3 + far + 8.0) * 2.0 ** -23 * far
    tol = (a.abs() + ea) * eu + ea * u.abs()
    h = gated.forward(G, U, x)
    close(h, a * u, tol + HALF[dtype] * ((a * u).abs() + tol) + LEAST[dtype])
    assert torch.equal(h, gated.forward(G, U, x))
