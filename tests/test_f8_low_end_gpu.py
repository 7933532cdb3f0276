"""8-bit matrices at the low end of fp32's range, on the GPU: values read back
are exact or rounded once; in products, values, products and sums below 2^-126
count as they are or as zero.

Bounds of a product: test_f8_gpu.py's, and the terms with a factor below
2^-126, and 2^-126 for each of k sums."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import f8
from oracle import f8_oracle as fo
from test_f8_gpu import HALF, as64, normal, reference

pytestmark = pytest.mark.gpu

LOW = 2.0 ** -126


@pytest.mark.parametrize("kind", [f8.WEIGHT, f8.ROWS])
def test_every_code_at_the_lowest_scales(kind):
    table = np.concatenate([fo.e4m3_table()[:127], -fo.e4m3_table()[:127]])
    for e in range(-127, -116):
        want = np.resize(table, (16, 256)) * 2.0 ** e
        want[:, ::128] = 448.0 * 2.0 ** e
        a = torch.from_numpy(want).float().cuda()
        assert np.array_equal(as64(a), want)
        Q = f8.pack(a) if kind == f8.WEIGHT else f8.quant(a)
        assert bool((Q.scales.view(-1, 4)[:, :2] == e + 127).all())
        assert np.array_equal(as64(f8.unpack(Q)), want)
        got = as64(f8.unpack(Q, out_dtype=torch.bfloat16))
        assert np.array_equal(got, as64(torch.from_numpy(want).to(torch.bfloat16)))
        exact = np.abs(want) >= 2.0 ** -130
        assert np.array_equal(got[exact], want[exact])


@pytest.mark.parametrize("m", [1, 3, 20, 200, 600])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ew,ex", [(-110, 100), (-120, 110), (-124, 120), (-128, 120), (-133, 125), (-60, -60), (100, -124)])
def test_products_of_values_near_the_lowest(m, out, ew, ex):
    n, k = 300, 700
    w = normal(1, n, k, "f32") * 2.0 ** ew
    x = normal(2, m, k, "f32") * 2.0 ** ex
    ref, s = reference(x, w)
    xv, wv = fo.values(*fo.quantise(as64(x), 1)), fo.values(*fo.quantise(as64(w), 128))
    lost = np.where(np.abs(xv) < LOW, np.abs(xv), 0.0) @ np.abs(wv).T \
        + np.abs(xv) @ np.where(np.abs(wv) < LOW, np.abs(wv), 0.0).T
    tol = k * 2.0 ** -23 * s[0] + HALF[out] * np.abs(ref) + lost + k * LOW
    if out != torch.float32:
        tol += 2.0 ** -11 * s[1]
    y = as64(f8.gemm(f8.pack(w), x, out_dtype=out))
    assert np.all(np.abs(y - ref) <= tol), (float(np.max(np.abs(y - ref) - tol)), float(np.abs(ref).max()))
    if min(ew, ex) >= -110:
        assert lost.max() < 0.01 * np.abs(ref).max()    # (so that the bound says something there)
