"""Each gradient of the cross entropy alone is bit for bit what both together
are, where most of the head is padding (dX works through the vocabulary, dW
through every row) and the logits go through the library's product."""
import pytest
import torch

from matmul_pack_b1_amd import xent
from test_xent_gpu import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sparse", [0.0, 0.5])
@pytest.mark.parametrize("m,n,n_vocab,k,tile,dtype", [
    (9, 8448, 2000, 2048, 256, "f16"), (16, 8448, 3000, 2048, 64, "f16"), (40, 8448, 1000, 2048, 64, "f16"),
    (40, 8448, 1, 256, 64, "bf16"), (64, 16384, 900, 256, 128, "bf16"), (3, 4096, 65, 256, 64, "f16"),
    (200, 2048, 130, 256, 64, "bf16")])
def test_one_gradient_is_the_same_as_both(m, n, n_vocab, k, tile, dtype, sparse):
    P, w, x, target, grad = make(n, k, m, n_vocab, dtype, tile=(tile, tile), sparse=sparse, seed=m, sigma=0.05)
    loss, lse, dx, dw = check(P, w, x, target, grad, n_vocab)   # compares each alone with both
    assert bool((dw[n_vocab:] == 0).all())
    again = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dw=True)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
