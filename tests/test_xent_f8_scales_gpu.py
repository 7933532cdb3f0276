"""Gradient of the input over an 8-bit head whose blocks' scales lie up to 2^30
apart: bounds as in test_xent_gpu.py, and for fp16 2^-31 of the largest scale
for every entry of W' in a block more than 2^21 below it."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import f8, xent
from oracle import f8_oracle as fo
from test_xent_gpu import DT, as64, bounds, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", [(10, 700), (100, 700), (100, 8576), (300, 8576)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("drops", [(0, 8, 15, 21), (0, 22, 26, 30), (30, 0, 24, 10)])
def test_blocks_of_far_apart_scales(m, n, dtype, drops):
    k = 500
    g = torch.Generator().manual_seed(m + n)
    w = torch.randn(n, k, generator=g) * 2.0 ** 4
    x = torch.randn(m, k, generator=g) * 2.0 ** -6
    for i, d in enumerate(drops):
        w[:, 128 * i:128 * (i + 1)] *= 2.0 ** -d
    w = w.cuda()                                # fp32: fp16 would not hold the smallest
    x = x.to(DT[dtype]).cuda()
    target = torch.randint(0, n, (m,), generator=g).cuda()
    grad = (torch.randn(m, generator=g) * 2.0 ** 10).cuda()
    codes, exps = fo.quantise(as64(w), 128)
    xv, wv = fo.values(*fo.quantise(as64(x), 1)), fo.values(codes, exps)
    (loss, lse, dx, _), (tol_loss, _, tol_dx, _) = bounds(xv, wv, x, target, grad, n, k)
    P = f8.pack(w)
    got_loss, got_lse = xent.loss(P, x, target)
    within("loss", got_loss, loss, tol_loss)
    got, _ = xent.backward(P, x, target, got_lse, grad)
    if dtype == "f16":
        z = xv @ wv.T
        dz = np.exp(z - lse[:, None])
        dz[np.arange(m), target.cpu().numpy()] -= 1.0
        top = exps.max()
        off = np.where(np.repeat(exps < top - 21, 128, axis=1)[:, :k], 2.0 ** (top - 31.0), 0.0)
        tol_dx = tol_dx + np.abs(dz * as64(grad)[:, None]) @ off
    # fp16 ends at 65504 and rounds to an infinity from 65520 on: where the bound
    # reaches beyond 65504, either is right
    beyond = np.abs(dx) + tol_dx > torch.finfo(x.dtype).max
    v = as64(got)
    ok = (v == np.sign(dx) * np.inf) | (np.abs(v - dx) <= tol_dx)
    assert beyond.mean() < 0.02 and ok[beyond].all()
    within("dx", torch.from_numpy(np.where(beyond, dx, v)), dx, tol_dx)
    small = int(np.argmax(drops))               # the bound says something of the smallest block too
    cols = slice(128 * small, min(k, 128 * (small + 1)))
    if drops[small] <= 26 or dtype == "bf16":
        assert tol_dx[:, cols].max() < 0.1 * np.abs(dx[:, cols]).max()


@pytest.mark.parametrize("pad", [0, 1, 63, 100, 300, 8000])
@pytest.mark.parametrize("m,dtype", [(9, "f16"), (100, "bf16"), (300, "f16")])
def test_vocabulary_ends_anywhere(m, dtype, pad):
    """Padding rows of NaN (a block's scale leaves them out), workspaces of NaN
    bytes."""
    n, k = 8450, 333
    n_vocab = n - pad
    g = torch.Generator().manual_seed(m + pad)
    w = (torch.randn(n, k, generator=g) * 0.1).to(DT[dtype])
    w[n_vocab:] = float("nan")
    x = torch.randn(m, k, generator=g).to(DT[dtype]).cuda()
    target = torch.randint(0, n_vocab, (m,), generator=g)
    target[::5] = -100
    target, grad = target.cuda(), (torch.randn(m, generator=g) / m).cuda()
    P = f8.pack(w.cuda())
    xv = fo.values(*fo.quantise(as64(x), 1))
    wv = np.nan_to_num(fo.values(*fo.quantise(as64(w), 128)))
    want, tol = bounds(xv, wv, x, target, grad, n_vocab, k)

    def workspace(**what):
        return torch.full((xent.workspace_bytes(P, m, **what),), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = xent.loss(P, x, target, n_vocab=n_vocab, workspace=workspace())
    dx, _ = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, workspace=workspace(dx=True))
    for name, got, ref, lim in zip(("loss", "lse", "dx"), (loss, lse, dx), want, tol):
        within(name, got, ref, lim)
