"""G, U and H of the gated projection in rows apart, at any element-aligned address
(include/hyb_gated.h), on each of its routes: the same bits as in dense rows, and
nothing written between them.  The binding gives dense G and U only."""
import ctypes

import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated

pytestmark = pytest.mark.gpu


def normal(seed, rows, cols, dtype, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(dtype)


def rows_apart(m, n, pitch, offset, dtype):
    base = torch.full((m * pitch + offset + 9,), 7.0, dtype=dtype, device="cuda")
    return base, torch.as_strided(base, (m, n), (pitch, 1), offset)


# decode, grouped decode, the matrix-core products, tiles whole and tiles cut
@pytest.mark.parametrize("n,k,m", [(192, 320, 1), (192, 320, 4), (192, 320, 9), (192, 320, 16), (192, 320, 40),
                                   (192, 320, 100), (320, 192, 133), (64, 768, 129)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_kept_products(n, k, m, dtype):
    tiles = (torch.arange(n // 64 * (k // 64)) % 2).to(torch.uint8).numpy()
    P, Q = (hb.pack(normal(i, n, k, dtype, k ** -0.5), tiles, 64, 64, "idx2") for i in (1, 2))
    x = normal(3, m, k, dtype)
    want = gated.forward(P, Q, x, save=True)
    pair, _, _ = gated._pair(P, Q)
    ws = torch.full((max(gated.workspace_bytes(P, Q, m), 16),), 255, dtype=torch.uint8, device="cuda")
    for step, offset in ((1, 1), (3, 2), (4, 4), (6, 3)):
        bases, views = zip(rows_apart(m, n, n + step, offset, dtype), rows_apart(m, n, n + step + 1, offset, torch.float32),
                           rows_apart(m, n, n + step + 2, offset + 1, torch.float32))
        h, g, u = views
        st = gated.lib().hyb_gated(ctypes.byref(pair), gated.ACTS["silu"], x.data_ptr(),
                                   {torch.bfloat16: hb.HYB_BF16, torch.float16: hb.HYB_F16}[dtype], m, k,
                                   h.data_ptr(), h.stride(0), g.data_ptr(), g.stride(0), u.data_ptr(), u.stride(0),
                                   ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        hb.check(st, "hyb_gated")
        for got, ref in zip(views, want):
            assert torch.equal(got, ref)
            got.fill_(7.0)
        assert all(bool((b == 7.0).all()) for b in bases)
