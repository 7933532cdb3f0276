"""The 4-bit product at the largest rows and columns that hyb_q4.h allows.

Weights and activations are small whole numbers (codes of scale 1), so that sums of up
to 2^24 are exact."""
import pytest
import torch

from matmul_pack_b1_amd import q4

pytestmark = pytest.mark.gpu


def whole_numbers(rows, k, seed):
    """-2 .. 2, and a 6 in every group: the scale is 1."""
    g = torch.Generator("cuda").manual_seed(seed)
    w = torch.randint(-2, 3, (rows, k), generator=g, device="cuda", dtype=torch.int8)
    w[:, ::32] = 6
    return w.to(torch.bfloat16)


def ones(m, k, seed, few):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randint(-1, 2, (m, k), generator=g, device="cuda", dtype=torch.int8)
    return (x * (torch.rand(k, generator=g, device="cuda") < few)).to(torch.bfloat16)


@pytest.mark.parametrize("m", [1, 4, 13, 40, 300])
def test_longest_rows(m):
    n, k = 19, 1 << 22
    w = whole_numbers(n, k, 1)
    Q = q4.pack(w)
    x = ones(m, k, m, 0.01)
    want = x.double() @ w.double().t()
    assert float((x.double().abs() @ w.double().abs().t()).max()) < 1 << 24
    assert torch.equal(q4.gemm(Q, x).double(), want)
    assert torch.equal(q4.gemm(Q, x.half()).double(), want)
    assert torch.equal(q4.unpack(Q), w)


@pytest.mark.parametrize("m", [1, 3, 20])
def test_most_rows(m):
    n, k = (1 << 27) - 16, 32
    w = whole_numbers(n, k, 2)
    Q = q4.pack(w)
    x = ones(m, k, m, 1.0)
    y = q4.gemm(Q, x)
    for r in range(0, n, 1 << 24):
        assert torch.equal(y[:, r:r + (1 << 24)], x.float() @ w[r:r + (1 << 24)].float().t())
    del y
    assert torch.equal(q4.unpack(Q), w)
