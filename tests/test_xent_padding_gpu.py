"""Cross entropy over packed heads whose vocabulary ends anywhere in a tile row,
or tile rows before the end: padding rows of NaN, workspaces of NaN bytes."""
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import xent
from test_xent_gpu import as64, bounds, make, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pad", [0, 1, 64, 100, 255, 256, 300, 8000])
@pytest.mark.parametrize("m,tile,dtype,sparse", [(9, 64, "bf16", 0.0), (9, 256, "f16", 0.0), (100, 64, "f16", 0.0),
                                                 (100, 128, "bf16", 0.0), (300, 256, "bf16", 0.0), (300, 64, "bf16", 0.0),
                                                 (9, 256, "bf16", 0.5), (300, 128, "f16", 0.5)])
def test_vocabulary_ends_anywhere(m, tile, dtype, sparse, pad):
    n, k = 8448, 256
    n_vocab = n - pad
    _, w, x, target, grad = make(n, k, m, n_vocab, dtype, seed=pad + m)
    w[n_vocab:] = float("nan")
    tmap = (torch.rand(n // tile, k // tile, generator=torch.Generator().manual_seed(3)) < sparse)
    P = hb.pack(w, tmap.to(torch.uint8).numpy(), tile, tile)
    wv = as64(hb.unpack(P))
    wv[n_vocab:] = 0.0
    want, tol = bounds(as64(x), wv, x, target, grad, n_vocab, k)

    def workspace(**what):
        return torch.full((xent.workspace_bytes(P, m, **what),), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = xent.loss(P, x, target, n_vocab=n_vocab, workspace=workspace())
    dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dw=True, workspace=workspace(dx=True, dw=True))
    for name, got, ref, lim in zip(("loss", "lse", "dx", "dw"), (loss, lse, dx, dw), want, tol):
        within(name, got, ref, lim)
    one, _ = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, workspace=workspace(dx=True))
    _, two = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dx=False, need_dw=True,
                           workspace=workspace(dw=True))
    assert torch.equal(one, dx) and torch.equal(two, dw) and bool((dw[n_vocab:] == 0).all())
