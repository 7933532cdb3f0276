"""Cross entropy over a packed head whose tile index names no slot for some
tiles, in a workspace of NaN bytes: the tiles count as zeros in the loss and in
both gradients, with and without padding and sparse tiles."""
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import xent
from test_xent_gpu import as64, bounds, make, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pad", [0, 12])
@pytest.mark.parametrize("sparse", [0.0, 0.5])
@pytest.mark.parametrize("m,n,tile", [(6, 512, 64), (100, 512, 256), (100, 8448, 64), (300, 8448, 256)])
def test_tiles_without_a_slot_are_zeros(m, n, tile, sparse, pad):
    k, n_vocab = 512, n - pad
    P, w, x, target, grad = make(n, k, m, n_vocab, "bf16", tile=(tile, tile), sparse=sparse, seed=31)
    wv = as64(hb.unpack(P))
    across = k // tile
    bad = [0, across + 1, (n // tile - 1) * across + 1]
    for b in bad:
        r, c = b // across * tile, b % across * tile
        wv[r:r + tile, c:c + tile] = 0.0
    P.tidx[torch.tensor(bad, device="cuda")] = P.layout.n_dense + 5
    want, tol = bounds(as64(x), wv, x, target, grad, n_vocab, k)

    def workspace(**what):
        return torch.full((xent.workspace_bytes(P, m, **what),), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = xent.loss(P, x, target, n_vocab=n_vocab, workspace=workspace())
    dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dw=True,
                           workspace=workspace(dx=True, dw=True))
    one, _ = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, workspace=workspace(dx=True))
    for name, got, ref, lim in zip(("loss", "lse", "dx", "dw", "dx alone"), (loss, lse, dx, dw, one),
                                   (*want, want[2]), (*tol, tol[2])):
        within(name, got, ref, lim)
