"""Cross entropy of finite logits far beyond any a healthy model has, on the
GPU: the loss and the gradients stay those of the formula on every route.

The logits are exact: row v of the head holds the five base-8 digits of v (the
same for all 12 copies of five columns), a token's x the powers of 8 times
+-2^e, so z = +-12 v 2^e sums integers below 2^24 without a rounding and the
largest is alone.  From 2^e = 2^5 on, its neighbours lie 384 below: softmax is
one-hot to the last bit.  In between are tokens that see digit 0 alone, with
logits 0..7.

Bounds: lse and loss 2^-22 |lse| (logarithm, its sum with the maximum, the
difference from the target's logit) + 2^-17 (exponentials and their sums);
dz as in test_xent_gpu.py with exact logits: h |dz| + 2^-17 p, and 2^-22 |lse| p
for the tokens of small logits (lse of the large ones is the largest logit,
exact)."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import f8, xent
from oracle import xent_oracle as xo
from test_xent_gpu import DT, HALF, TINY, as64, operands, within

pytestmark = pytest.mark.gpu

K, COPIES = 64, 12


def make(n, m, n_vocab, dtype, head, exponents, lift):
    g = torch.Generator().manual_seed(m + n)
    order = torch.randperm(n, generator=g)
    digits = torch.stack([(order >> (3 * j)) & 7 for j in range(5)], 1).double()
    w = torch.zeros(n, K, dtype=torch.float64)
    w[:, :5 * COPIES] = digits.repeat(1, COPIES) * 2.0 ** lift
    x = torch.zeros(m, K, dtype=torch.float64)
    powers = torch.tensor([8.0 ** j for j in range(5)], dtype=torch.float64).repeat(COPIES)
    for t in range(m):
        e = exponents[t % len(exponents)]
        if e is None:
            x[t, 0] = 2.0 ** -lift
        else:
            x[t, :5 * COPIES] = powers * 2.0 ** (e - lift) * (-1.0 if t % 2 else 1.0)
    w, x = w.to(DT[dtype]).cuda(), x.to(DT[dtype]).cuda()
    target = torch.randint(0, n_vocab, (m,), generator=g)
    target[::7] = -100
    grad = (torch.randn(m, generator=g) / m).cuda()
    P = hb.pack(w, np.zeros((n // 64, 1), np.uint8), 64, 64) if head == "packed" else f8.pack(w)
    return P, w, x, target.cuda(), grad


@pytest.mark.parametrize("head,dtype,lift,exponents", [
    ("packed", "bf16", 0, (None, 9, 13, 18, 27, 60, 100)), ("packed", "bf16", 0, (27,)),
    ("packed", "f16", 13, (None, 9, 13, 16)), ("f8", "bf16", 0, (None, 9, 13, 18, 27, 60, 100)),
    ("f8", "f16", 13, (None, 9, 13, 16)),
])
@pytest.mark.parametrize("m,n", [(5, 8576), (100, 512), (100, 8576), (300, 8576)])
def test_large_finite_logits(m, n, head, dtype, lift, exponents):
    n_vocab = n - 12
    P, w, x, target, grad = make(n, m, n_vocab, dtype, head, exponents, lift)
    xv, wv = operands(P, w, x)
    assert np.array_equal(xv, as64(x)) and np.array_equal(wv, as64(w))
    t, g, h = target.cpu().numpy(), as64(grad), HALF[x.dtype]
    loss, lse, dx, dw = xo.cross_entropy(xv, wv, t, n_vocab, grad=g)
    got_loss, got_lse = xent.loss(P, x, target, n_vocab=n_vocab)
    tol = 2.0 ** -17 + 2.0 ** -22 * np.abs(lse)
    within("lse", got_lse, lse, tol)
    within("loss", got_loss, loss, tol + 2.0 ** -24 * np.abs(loss))
    seen = t != -100
    # (ignored tokens have lse 0: their z is taken as 0, else exp z * 0 is inf * 0)
    p = np.exp(np.where(seen[:, None], xv, 0.0) @ wv[:n_vocab].T - lse[:, None]) * seen[:, None]
    G = p.copy()
    G[np.flatnonzero(seen), t[seen]] -= 1.0
    soft = np.where(np.abs(lse) < 64, 2.0 ** -22 * np.abs(lse), 0.0)
    ep = np.abs(G) * h + p * (2.0 ** -17 + soft)[:, None]
    low = 2 * (2.0 ** -39 if dtype == "f16" else 2.0 ** -126) * np.abs(g[seen]).max()
    packed = head == "packed"
    got_dx, got_dw = xent.backward(P, x, target, got_lse, grad, n_vocab=n_vocab, need_dw=packed)
    eg = ((ep + np.abs(G) * n_vocab * 2.0 ** -23) * np.abs(g)[:, None] + low) * seen[:, None]
    within("dx", got_dx, dx, eg @ np.abs(wv[:n_vocab]) + h * np.abs(dx) + TINY[x.dtype])
    if packed:
        eg = ((ep + np.abs(G) * m * 2.0 ** -23) * np.abs(g)[:, None] + low) * seen[:, None]
        tol_dw = np.zeros_like(wv)
        tol_dw[:n_vocab] = eg.T @ np.abs(xv)
        within("dw", got_dw, dw, tol_dw + h * np.abs(dw) + TINY[x.dtype])
