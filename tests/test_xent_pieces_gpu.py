"""Cross entropy over heads that take more than one piece, in the loss or in the
gradients, on every route: each test first asks the library that it does."""
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import xent
from test_xent_gpu import check, make

pytestmark = pytest.mark.gpu


def pieces(P, m, **what):
    return -(-P.shape[0] // xent.piece_rows(P, m, **what))


# (m, n, n_vocab): the last piece shorter than the parts of dX; the vocabulary
# ending within a piece with pieces of padding behind; within the first piece
MANY = [(1000, 66048, 66001), (1000, 98560, 65000), (1000, 66048, 32768), (1000, 66048, 100)]
# pieces grow for few tokens: tiles of 128 tokens, and the library's product
FEW = [(100, 270080, 270001), (16, 600064, 600001)]


@pytest.mark.parametrize("m,n,n_vocab", MANY + FEW)
@pytest.mark.parametrize("head,dtype,tile,meta,sparse", [
    ("packed", "bf16", (64, 64), "idx2", 0.0), ("packed", "f16", (128, 64), "mask4", 0.5), ("f8", "bf16", None, None, 0.0)])
def test_gradients_of_many_pieces(m, n, n_vocab, head, dtype, tile, meta, sparse):
    if tile is not None:
        n = n // tile[0] * tile[0]
    P, w, x, target, grad = make(n, 64, m, n_vocab, dtype, head=head, tile=tile, meta=meta, seed=m + n, sparse=sparse)
    assert pieces(P, m, dx=True) >= 2
    if head == "packed":
        assert pieces(P, m, dx=True, dw=True) >= 2 and pieces(P, m, dw=True) >= 2
    check(P, w, x, target, grad, n_vocab)


@pytest.mark.parametrize("m", [16, 1000])
def test_fp16_gradient_of_an_8_bit_head_of_many_pieces(m):
    n = 600064 if m == 16 else 66048
    P, w, x, target, grad = make(n, 64, m, n - 47, "f16", head="f8", seed=41)
    assert pieces(P, m, dx=True) >= 2
    check(P, w, x, target, grad, n - 47)


@pytest.mark.parametrize("m", [200, 600])
def test_loss_of_many_pieces(m):
    """Over sparse tiles: through the product (few tokens) and from expanded
    tiles."""
    n, n_vocab = 66048, 65900
    P, w, x, target, grad = make(n, 128, m, n_vocab, "bf16", seed=42)
    assert pieces(P, m) >= 2
    check(P, w, x, target, grad, n_vocab)


def test_pieces_at_two_sizes_of_the_vocabulary_are_the_same_bits():
    """Entries behind the vocabulary change nothing, piece by piece."""
    m, n, n_vocab = 1000, 98304, 33000
    P, w, x, target, grad = make(n, 64, m, n_vocab, "bf16", seed=43)
    tmap = (P.tidx[:33024 // 64].view(-1, 1) < 0).to(torch.uint8).cpu().numpy()
    small = hb.pack(w[:33024], tmap, 64, 64)
    assert pieces(P, m, dx=True) == 3 and pieces(small, m, dx=True) == 2
    loss, lse = xent.loss(P, x, target, n_vocab=n_vocab)
    loss2, lse2 = xent.loss(small, x, target, n_vocab=n_vocab)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dw=True)
    dx2, dw2 = xent.backward(small, x, target, lse, grad, n_vocab=n_vocab, need_dw=True)
    assert torch.equal(dx, dx2) and torch.equal(dw[:33024], dw2) and bool((dw[n_vocab:] == 0).all())
