"""Cross entropy over a vocabulary projection on the GPU against the float64
oracle.

Bounds, from the rounding steps of the calculation (h is half a step of the
16-bit type: 2^-8 bf16, 2^-11 fp16):
  z     fp32 sums of exact products: ez = k 2^-23 max_v sum_c |x w|
  loss  2 ez; exponentials and their fp32 sums, at most 2^-17 of the sum (about
        a hundred roundings), and the roundings of lse and z: 2^-22 |lse|
  dX    each entry of dz = grad (softmax - onehot) is off by h |dz| (its
        rounding, plus, over the largest |grad| rounded up to a power of two,
        2^-39 where fp16 scaled by 2^14 is subnormal, and 2^-126 in any type:
        the exponential's result and a matrix operand below the smallest
        normal fp32 or bf16 number count as zero) and |grad| p (ez + 2^-17);
        fp32 sums n_vocab 2^-23; the result's own rounding h
  dW    the same with X in place of W and m in place of n_vocab"""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import f8, xent
from oracle import f8_oracle as fo
from oracle import xent_oracle as xo

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def as64(t):
    return t.detach().cpu().double().numpy()


def make(n, k, m, n_vocab, dtype, head="packed", tile=(64, 64), meta="idx2", seed=0, sigma=0.1, scale=1.0, sparse=0.5):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(n, k, generator=g) * sigma).to(DT[dtype]).cuda()
    x = (torch.randn(m, k, generator=g) * scale).to(DT[dtype]).cuda()
    target = torch.randint(0, n_vocab, (m,), generator=g)
    target[torch.rand(m, generator=g) < 0.2] = -100
    grad = torch.randn(m, generator=g) / max(m, 1)
    if head == "packed":
        tmap = (torch.rand(n // tile[0], k // tile[1], generator=g) < sparse).to(torch.uint8).numpy()
        P = hb.pack(w, tmap, *tile, meta)
    else:
        P = f8.pack(w)
    return P, w, x, target.cuda(), grad.cuda()


def operands(P, w, x):
    """x and W' as the calculation sees them, float64."""
    if isinstance(P, hb.PackedWeight):
        return as64(x), as64(hb.unpack(P))
    return fo.values(*fo.quantise(as64(x), 1)), fo.values(*fo.quantise(as64(w), 128))


def bounds(xv, wv, x, target, grad, n_vocab, k):
    """(loss, lse, dx, dw) of the oracle, and the four error bounds."""
    t, g = target.cpu().numpy(), as64(grad)
    h, tiny = HALF[x.dtype], TINY[x.dtype]
    sub = 2.0 ** -39 if x.dtype == torch.float16 else 2.0 ** -126
    loss, lse, dx, dw = xo.cross_entropy(xv, wv, t, n_vocab, grad=g)
    seen = (t != -100) & (t >= 0) & (t < n_vocab)
    xs, ws = np.where(seen[:, None], np.abs(xv), 0.0), np.abs(wv[:n_vocab])
    ez = k * 2.0 ** -23 * (xs @ ws.T).max(axis=1)
    tol_loss = 2 * ez + 2.0 ** -17 + 2.0 ** -22 * np.abs(lse)
    z = np.where(seen[:, None], xv, 0.0) @ wv[:n_vocab].T
    p = np.exp(z - lse[:, None]) * seen[:, None]
    G = p.copy()
    G[np.flatnonzero(seen), t[seen]] -= 1.0
    ag = np.abs(g)[:, None]
    low = 2 * sub * np.abs(g[seen]).max(initial=0.0)
    eg = ((np.abs(G) * (h + n_vocab * 2.0 ** -23) + p * (ez + 2.0 ** -17)[:, None]) * ag + low) * seen[:, None]
    tol_dx = eg @ ws + h * np.abs(dx) + tiny
    eg = ((np.abs(G) * (h + len(t) * 2.0 ** -23) + p * (ez + 2.0 ** -17)[:, None]) * ag + low) * seen[:, None]
    tol_dw = np.zeros_like(wv)
    tol_dw[:n_vocab] = eg.T @ xs
    tol_dw += h * np.abs(dw) + tiny
    return (loss, lse, dx, dw), (tol_loss, tol_loss, tol_dx, tol_dw)


def within(name, got, want, tol):
    err = np.abs(as64(got) - want)
    bad = ~(err <= tol)
    print(name, "worst error over bound", float(np.max(err / tol)) if err.size else 0.0)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(err[bad][0]), float(tol[bad][0]))


def check(P, w, x, target, grad, n_vocab):
    xv, wv = operands(P, w, x)
    want, tol = bounds(xv, wv, x, target, grad, n_vocab, x.shape[1])
    loss, lse = xent.loss(P, x, target, n_vocab=n_vocab)
    within("loss", loss, want[0], tol[0])
    within("lse", lse, want[1], tol[1])
    packed = isinstance(P, hb.PackedWeight)
    dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dw=packed)
    within("dx", dx, want[2], tol[2])
    if packed:
        within("dw", dw, want[3], tol[3])
        # each gradient alone is the same
        one, none = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab)
        assert none is None and torch.equal(one, dx)
        none, one = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dx=False, need_dw=True)
        assert none is None and torch.equal(one, dw)
    return loss, lse, dx, dw


@pytest.mark.parametrize("m", [1, 3, 16, 17, 40, 64, 65, 130, 256, 300])
@pytest.mark.parametrize("n,k,n_vocab", [(64, 64, 1), (256, 128, 250), (1024, 320, 1003), (1088, 192, 1088)])
def test_packed_head(m, n, k, n_vocab):
    check(*make(n, k, m, n_vocab, "bf16", seed=m + n), n_vocab)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tile,meta", [((64, 64), "idx2"), ((128, 128), "mask4"), ((256, 256), "idx2"),
                                       ((64, 256), "mask8"), ((256, 64), "mask4"), ((128, 128), "mask8")])
@pytest.mark.parametrize("m", [9, 200])
def test_packed_forms(m, dtype, tile, meta):
    check(*make(768, 512, m, 700, dtype, tile=tile, meta=meta, seed=m), 700)


@pytest.mark.parametrize("sparse", [0.0, 1.0])
@pytest.mark.parametrize("tile", [(64, 64), (64, 256), (128, 128), (256, 64), (256, 256)])
@pytest.mark.parametrize("m", [7, 70, 300])
def test_heads_of_one_kind_of_tile(m, tile, sparse):
    """No sparse tile: the dense stream is multiplied where it lies (but for
    the piece that holds padding); no dense one."""
    check(*make(1536, 768, m, 1536, "bf16", tile=tile, sparse=sparse, seed=m), 1536)
    check(*make(1536, 512, m, 1400, "f16", tile=tile, sparse=sparse, seed=m), 1400)


def test_dense_head_of_many_pieces():
    check(*make(66048, 64, 70, 66000, "bf16", sparse=0.0, seed=1), 66000)
    check(*make(66048, 320, 40, 66048, "bf16", sparse=0.0, seed=2), 66048)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 5, 33, 64, 65, 200, 300])
@pytest.mark.parametrize("n,k,n_vocab", [(1, 1, 1), (300, 200, 300), (1003, 333, 1000), (640, 1024, 513)])
def test_f8_head(m, n, k, n_vocab, dtype):
    check(*make(n, k, m, n_vocab, dtype, head="f8", seed=m + n), n_vocab)


@pytest.mark.parametrize("head", ["packed", "f8"])
@pytest.mark.parametrize("m", [20, 70])
def test_many_pieces(m, head):
    """More entries than one piece holds (32768), the last piece ragged."""
    n, n_vocab = 70016, 69999
    check(*make(n, 64, m, n_vocab, "bf16", head=head, seed=m), n_vocab)


def test_many_tokens():
    """Few entries per piece because of many tokens; more than 256 tiles."""
    check(*make(1024, 64, 20000, 1000, "bf16", seed=3), 1000)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("head", ["packed", "f8"])
@pytest.mark.parametrize("m,n", [(10, 512), (150, 512), (150, 8448)])
def test_confident_and_flat_rows(m, n, head, dtype):
    """Logits of +-hundreds (softmax one-hot, probabilities far below the
    smallest 16-bit number) and all equal (x = 0)."""
    P, w, x, target, grad = make(n, 256, m, n - 12, dtype, head=head, seed=4, scale=40.0)
    x[0] = 0.0
    target[0] = 7
    check(P, w, x, target, grad, n - 12)


@pytest.mark.parametrize("head", ["packed", "f8"])
@pytest.mark.parametrize("m,n", [(6, 512), (100, 512), (100, 8576)])
def test_masked_places_are_not_looked_at(m, n, head):
    """NaN and infinities in ignored tokens' x and grad and in the head's
    padding rows change nothing."""
    k, n_vocab = 256, n - 128       # padding from a block of 128 on
    P, w, x, target, grad = make(n, k, m, n_vocab, "bf16", head=head, seed=5)
    target[1], target[3] = -100, -100
    want = check(P, w, x, target, grad, n_vocab)
    x2, grad2, w2 = x.clone(), grad.clone(), w.clone()
    x2[1], x2[3] = float("nan"), float("inf")
    grad2[1], grad2[3] = float("nan"), float("inf")
    w2[n_vocab:] = float("nan")
    w2[n_vocab + 1:, ::2] = float("inf")
    if head == "packed":
        P2 = hb.pack(w2, np.zeros((n // 64, k // 64), np.uint8), 64, 64, "idx2")
        P = hb.pack(w, np.zeros((n // 64, k // 64), np.uint8), 64, 64, "idx2")
        want = check(P, w, x, target, grad, n_vocab)
    else:
        P2 = f8.pack(w2)
    loss, lse = xent.loss(P2, x2, target, n_vocab=n_vocab)
    dx, dw = xent.backward(P2, x2, target, lse, grad2, n_vocab=n_vocab, need_dw=head == "packed")
    for got, ref in zip((loss, lse, dx, dw), want):
        if ref is not None:
            assert torch.equal(got, ref)
    assert float(loss[1]) == 0 and float(lse[3]) == 0 and bool((dx[1] == 0).all())


@pytest.mark.parametrize("m,n", [(6, 512), (100, 512), (100, 8448)])
def test_all_tokens_ignored(m, n):
    P, w, x, target, grad = make(n, 128, m, n - 12, "bf16", seed=6)
    target.fill_(-100)
    x.fill_(float("nan"))
    loss, lse = xent.loss(P, x, target, n_vocab=n - 12)
    dx, dw = xent.backward(P, x, target, lse, grad * float("nan"), n_vocab=n - 12, need_dw=True)
    for t in (loss, lse, dx, dw):
        assert bool((t == 0).all())


@pytest.mark.parametrize("head", ["packed", "f8"])
@pytest.mark.parametrize("m,n", [(6, 512), (100, 512), (100, 8448)])
def test_bad_targets_are_nan(m, n, head):
    P, w, x, target, grad = make(n, 128, m, n - 12, "bf16", head=head, seed=7)
    ok = check(P, w, x, target, grad, n - 12)
    target[0], target[2], target[4] = n - 12, -1, 2 ** 40
    loss, lse = xent.loss(P, x, target, n_vocab=n - 12)
    dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n - 12, need_dw=head == "packed")
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    bad[[0, 2, 4]] = True
    assert bool(loss[bad].isnan().all()) and bool(dx[bad].isnan().all())
    assert torch.equal(loss[~bad], ok[0][~bad]) and torch.equal(dx[~bad], ok[2][~bad])
    if dw is not None:
        assert bool(dw[:n - 12].isnan().all())
    other = torch.where(target == n - 12, torch.full_like(target, 99), target)
    assert bool((xent.loss(P, x, other, n_vocab=n - 12, ignore_index=2 ** 40)[0][[2]]).isnan().all())


@pytest.mark.parametrize("m,n", [(6, 512), (100, 512), (100, 8448)])
def test_nan_in_a_token_stays_there(m, n):
    P, w, x, target, grad = make(n, 128, m, n - 12, "bf16", seed=8)
    target[:] = torch.arange(m) % 500
    loss, lse = xent.loss(P, x, target, n_vocab=n - 12)
    dx, _ = xent.backward(P, x, target, lse, grad, n_vocab=n - 12)
    x[2, 5] = float("nan")
    loss2, lse2 = xent.loss(P, x, target, n_vocab=n - 12)
    dx2, _ = xent.backward(P, x, target, lse2, grad, n_vocab=n - 12)
    rest = torch.arange(m, device="cuda") != 2
    assert bool(loss2[2].isnan()) and bool(dx2[2].isnan().all())
    assert torch.equal(loss2[rest], loss[rest]) and torch.equal(dx2[rest], dx[rest])


def test_ignore_index_and_default_vocabulary():
    P, w, x, target, grad = make(256, 128, 30, 256, "bf16", seed=9)
    a, lse = xent.loss(P, x, target)
    t2 = torch.where(target == -100, torch.full_like(target, 3), target)
    keep = t2 != 3
    b, _ = xent.loss(P, x, t2, ignore_index=3)
    assert torch.equal(a[keep], b[keep]) and bool((b[~keep] == 0).all())


@pytest.mark.parametrize("head", ["packed", "f8"])
def test_strides_and_given_outputs(head):
    n, k, m, n_vocab = 320, 192, 70, 311
    P, w, x, target, grad = make(n, k, m, n_vocab, "bf16", head=head, seed=10)
    _, lse, dx, dw = check(P, w, x, target, grad, n_vocab)
    wide = torch.full((m, k + 8), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, :k] = x
    loss2, lse2 = xent.loss(P, wide[:, :k], target, n_vocab=n_vocab)
    assert torch.equal(lse2, lse)
    for pad in (8, 5):
        gx = torch.full((m, k + pad), 7.0, dtype=x.dtype, device="cuda")
        gw = torch.full((n, k + pad), 7.0, dtype=x.dtype, device="cuda") if head == "packed" else None
        xent.backward(P, wide[:, :k], target, lse, grad, n_vocab=n_vocab, dx=gx[:, :k],
                      dw=gw[:, :k] if gw is not None else None)
        assert torch.equal(gx[:, :k], dx) and bool((gx[:, k:] == 7).all())
        if gw is not None:
            assert torch.equal(gw[:, :k], dw) and bool((gw[:, k:] == 7).all())


def test_empty_batch():
    P, w, x, target, grad = make(256, 128, 0, 256, "bf16", seed=11)
    loss, lse = xent.loss(P, x, target)
    assert loss.shape == (0,)
    dw = torch.full((256, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    dx, dw = xent.backward(P, x, target, lse, grad, dw=dw)
    assert dx.shape == (0, 128) and bool((dw == 0).all())


@pytest.mark.parametrize("scale", [2.0 ** -60, 1.0, 2.0 ** 40])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [256, 8448])
def test_gradients_of_any_size(dtype, scale, n):
    """dW's 16-bit operand carries grad: scaled by its largest magnitude."""
    P, w, x, target, grad = make(n, 128, 90, n - 6, "bf16", seed=12)
    if dtype == "f16":
        P, w, x, target, grad = make(n, 128, 90, n - 6, "f16", seed=12)
        scale = min(max(scale, 2.0 ** -6), 2.0 ** 6)     # what an fp16 gradient can hold
    check(P, w, x, target, grad * scale, n - 6)


@pytest.mark.parametrize("n", [512, 8448])
def test_gradient_against_differences(n):
    """Loss differences along single coordinates of x against dX: both sides'
    bounds and the cubic term of a central difference."""
    k, m, n_vocab, step = 128, 96, n - 12, 2.0 ** -3
    P, w, x, target, grad = make(n, k, m, n_vocab, "bf16", seed=13, sigma=0.25)
    x = (x * 16).round() / 16                     # x +- step stay exact
    x = x.clamp(-7, 7)
    xv, wv = operands(P, w, x)
    ones = torch.ones(m, device="cuda")
    (_, _, want, _), (tol_loss, _, tol_dx, _) = bounds(xv, wv, x, target, ones, n_vocab, k)
    _, lse = xent.loss(P, x, target, n_vocab=n_vocab)
    dx = as64(xent.backward(P, x, target, lse, ones, n_vocab=n_vocab)[0])
    for c in (0, 17, 127):
        hi, lo = x.clone(), x.clone()
        hi[:, c] += step
        lo[:, c] -= step
        diff = as64(xent.loss(P, hi, target, n_vocab=n_vocab)[0]) - as64(xent.loss(P, lo, target, n_vocab=n_vocab)[0])
        cubic = (step * np.abs(wv[:, c]).max() * 2) ** 3 / 3
        assert np.all(np.abs(diff - 2 * step * dx[:, c]) <= 3 * tol_loss + 2 * step * tol_dx[:, c] + cubic)
        assert np.abs(diff).max() > 10 * cubic


@pytest.mark.parametrize("head", ["packed", "f8"])
@pytest.mark.parametrize("m,n", [(5, 1024), (130, 1024), (130, 8448)])
def test_graph_replays(m, n, head):
    k, n_vocab = 256, n - 24
    P, w, x, target, grad = make(n, k, m, n_vocab, "bf16", head=head, seed=14)
    packed = head == "packed"

    def step():
        loss, lse = xent.loss(P, x, target, n_vocab=n_vocab)
        dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dw=packed)
        return [t for t in (loss, lse, dx, dw) if t is not None]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        _, _, x2, t2, g2 = make(n, k, m, n_vocab, "bf16", head=head, seed=20 + seed)
        x.copy_(x2)
        target.copy_(t2)
        grad.copy_(g2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_two_streams_and_repeats():
    """Calls on several streams at once, and again: the same bits."""
    sets = [make(1024, 256, m, 1000, "bf16", head=h, seed=15) for m, h in ((300, "packed"), (300, "f8"), (9, "packed"))]

    def step(P, w, x, target, grad):
        loss, lse = xent.loss(P, x, target, n_vocab=1000)
        dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=1000, need_dw=isinstance(P, hb.PackedWeight))
        return [t for t in (loss, lse, dx, dw) if t is not None]

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        for st, s, ref in zip(streams, sets, want):
            with torch.cuda.stream(st):
                got.append((step(*s), ref))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_together_a_frozen_8_bit_layer_under_an_8_bit_head():
    """hidden = x A^T (product), loss over the vocabulary, gradient back to
    hidden: the three operators in one run, against float64."""
    n, k, m, n_vocab = 900, 384, 150, 900
    g = torch.Generator().manual_seed(16)
    a = (torch.randn(k, 256, generator=g) * 0.1).to(torch.bfloat16).cuda()
    w = (torch.randn(n, k, generator=g) * 0.1).to(torch.bfloat16).cuda()
    x = torch.randn(m, 256, generator=g).to(torch.bfloat16).cuda()
    target = torch.randint(0, n_vocab, (m,), generator=g).cuda()
    grad = torch.full((m,), 1.0 / m, device="cuda")
    A, W = f8.pack(a), f8.pack(w)
    hidden = f8.gemm(A, x, out_dtype=torch.bfloat16)
    check(W, w, hidden, target, grad, n_vocab)
    ref = fo.values(*fo.quantise(as64(x), 1)) @ fo.values(*fo.quantise(as64(a), 128)).T
    assert np.all(np.abs(as64(hidden) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * np.abs(ref).max())


@pytest.mark.parametrize("sparse", [0.0, 0.5])
@pytest.mark.parametrize("m,n", [(6, 512), (100, 512), (100, 8448)])
def test_tile_index_out_of_range_adds_nothing(m, n, sparse):
    """Entries of the tile index that name no slot: their tiles count as
    zeros, as in the library's products."""
    P, w, x, target, grad = make(n, 256, m, n - 12, "bf16", tile=(64, 64), sparse=sparse, seed=17)
    tidx = P.tidx.clone()
    bad = torch.tensor([0, 5, 9, 30], device="cuda")
    for value in (P.layout.n_dense, -P.layout.n_sparse - 1, 2 ** 31 - 1, -2 ** 31):
        P.tidx.copy_(tidx)
        wv = as64(hb.unpack(P))
        for t in bad.tolist():
            r, c = t // 4, t % 4
            wv[r * 64:(r + 1) * 64, c * 64:(c + 1) * 64] = 0.0
        P.tidx[bad] = value
        want, tol = bounds(as64(x), wv, x, target, grad, n - 12, 256)
        loss, lse = xent.loss(P, x, target, n_vocab=n - 12)
        dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n - 12, need_dw=True)
        for name, got, ref, lim in zip(("loss", "lse", "dx", "dw"), (loss, lse, dx, dw), want, tol):
            within(name, got, ref, lim)


def test_tile_columns_beyond_one_register():
    """More than 64 tiles in a row, and more than 64 tile rows in a piece."""
    check(*make(128, 64 * 130, 70, 128, "bf16", seed=18, sigma=0.02), 128)
    check(*make(64 * 150, 128, 70, 64 * 150 - 3, "bf16", seed=19), 64 * 150 - 3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,h", [(5, 1024), (100, 1024), (300, 1024), (300, 8448)])
def test_logits_that_are_not_finite(m, h, dtype):
    """An entry at -inf has no share in the sum; one at +inf makes it +inf; a NaN
    makes it NaN; no entry above -inf gives -inf."""
    n, k = h - 424, 64
    _, w, x, target, _ = make(h, k, m, n, dtype, sparse=0.0, seed=m)
    x[:, 0] = x[:, 0].abs() + 0.5
    target[:] = torch.arange(m).cuda() % n
    w[3, 0] = w[n - 1, 0] = float("-inf")
    z = as64(x) @ np.nan_to_num(as64(w)[:n], neginf=0.0).T
    z[:, [3, n - 1]] = -np.inf
    top = z.max(1)
    want = top + np.log(np.exp(z - top[:, None]).sum(1))
    tol = 2 * k * 2.0 ** -23 * (np.abs(as64(x)) @ np.nan_to_num(np.abs(as64(w)[:n]), posinf=0.0).T).max(1) \
        + 2.0 ** -17 + 2.0 ** -22 * np.abs(want)
    none = np.zeros((h // 64, k // 64), np.uint8)

    def run(w):
        loss, lse = xent.loss(hb.pack(w, none, 64, 64), x, target, n_vocab=n)
        return as64(loss), as64(lse)
    loss, lse = run(w)
    within("lse", torch.from_numpy(lse), want, tol)
    assert loss[3] == np.inf and np.isfinite(np.delete(loss, [3])).all()
    w[400, 0] = float("inf")
    loss, lse = run(w)
    assert (lse == np.inf).all() and (np.delete(loss, [3]) == np.inf).all()
    w[400, 0] = float("nan")
    loss, lse = run(w)
    assert np.isnan(lse).all() and np.isnan(loss).all()
    w[:, 0] = float("-inf")
    loss, lse = run(w)
    assert (lse == -np.inf).all() and np.isnan(loss).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sparse", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("tile,meta", [((64, 64), "idx2"), ((128, 128), "mask8"), ((256, 256), "mask4"), ((64, 256), "idx2"),
                                       ((256, 64), "mask4")])
@pytest.mark.parametrize("m", [65, 129, 300, 600])
def test_packed_heads_of_many_tiles(m, tile, meta, sparse, dtype):
    """As many tiles as the logits need to be multiplied tile by tile."""
    check(*make(8448, 256, m, 8400, dtype, tile=tile, meta=meta, sparse=sparse, seed=m), 8400)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [65, 128, 200, 300])
@pytest.mark.parametrize("n,k,n_vocab", [(8449, 1, 8449), (8450, 333, 8321), (9000, 512, 8990)])
def test_8_bit_heads_of_many_tiles(m, n, k, n_vocab, dtype):
    check(*make(n, k, m, n_vocab, dtype, head="f8", seed=m + n), n_vocab)


def test_tile_columns_beyond_one_register_in_many_tiles():
    check(*make(8448, 64 * 70, 70, 8448, "bf16", seed=18, sigma=0.02), 8448)
    check(*make(64 * 150, 128, 70, 64 * 150 - 3, "bf16", seed=19), 64 * 150 - 3)
