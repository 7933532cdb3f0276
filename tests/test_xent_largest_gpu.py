"""Cross entropy at the ends of its range, on the GPU: 2^22 tokens, a head of
2^27 - 16 entries, a k of 2^21.  References in float64 on the GPU, in slices.

Bounds as in test_xent_gpu.py.  Where a sum has so many terms that the bound of
its fp32 additions (terms * 2^-23 of the sum of magnitudes) says nothing, the
terms' roundings are taken to add like independent ones, with a factor of 16:
an error 16 sqrt(terms) 2^-24 of the root of the sum of squares, or 16 h of it
for the 16-bit terms."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import f8, xent

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


def room(gib):
    free, _ = torch.cuda.mem_get_info()
    if free < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def test_most_tokens():
    room(40)
    m, n, n_vocab, k = 1 << 22, 256, 250, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    w = (torch.randn(n, k, generator=g, device="cuda") * 0.2).bfloat16()
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    target = torch.randint(0, n_vocab, (m,), generator=g, device="cuda")
    target[torch.rand(m, generator=g, device="cuda") < 0.1] = -100
    grad = torch.randn(m, generator=g, device="cuda") / 1024
    P = hb.pack(w, np.ones((n // 64, 1), np.uint8), 64, 64)
    loss, lse = xent.loss(P, x, target, n_vocab=n_vocab)
    dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dw=True)
    wv = hb.unpack(P).double()[:n_vocab]
    total, squares = torch.zeros(n_vocab, k, dtype=torch.float64, device="cuda"), 0.0
    for t0 in range(0, m, 1 << 20):
        s = slice(t0, t0 + (1 << 20))
        xs, seen = x[s].double(), target[s] != -100
        z = xs @ wv.t()
        ref = torch.logsumexp(z, 1)
        at = torch.where(seen, target[s], 0)[:, None]
        ez = k * 2.0 ** -23 * (xs.abs() @ wv.abs().t()).amax(1)
        tol = 2 * ez + 2.0 ** -17 + 2.0 ** -22 * ref.abs()
        assert bool(((loss[s] - torch.where(seen, ref - z.gather(1, at)[:, 0], 0.0)).abs() <= tol).all())
        assert bool(((lse[s] - torch.where(seen, ref, 0.0)).abs() <= tol).all())
        p = torch.exp(z - ref[:, None])
        G = p.scatter_add(1, at, torch.full_like(at, -1.0, dtype=torch.float64)) * seen[:, None]
        ag = grad[s].double().abs()[:, None]
        eg = (G.abs() * (H + n_vocab * 2.0 ** -23) + p * (ez + 2.0 ** -17)[:, None]) * ag * seen[:, None]
        dz = G * grad[s].double()[:, None]
        want = dz @ wv
        assert bool(((dx[s] - want).abs() <= eg @ wv.abs() + H * want.abs() + 2.0 ** -126).all())
        total += dz.t() @ xs
        squares = squares + (dz * dz).t() @ (xs * xs)
    tol = 16 * (H + m ** 0.5 * 2.0 ** -24) * squares.sqrt() + H * total.abs()
    assert bool(((dw[:n_vocab] - total).abs() <= tol).all()) and bool((dw[n_vocab:] == 0).all())
    assert float(tol.mean() / total.abs().mean()) < 0.2


@pytest.mark.parametrize("m", [2, 65])
def test_most_entries(m):
    room(64)
    n, k = (1 << 27) - 16, 1
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(n, k, generator=g, device="cuda")
    w[n - 5] = 9.0
    x = (torch.randn(m, k, generator=g, device="cuda") * 2).bfloat16()
    x[0] = 4.0                                      # the largest logit of token 0 is the entry n - 5
    target = torch.randint(0, n, (m,), generator=g, device="cuda")
    target[0], target[1] = n - 5, n - 1
    grad = torch.randn(m, generator=g, device="cuda")
    P, X = f8.pack(w), f8.unpack(f8.quant(x), out_dtype=torch.float32).double()
    wv = f8.unpack(P)[:, 0].double()
    del w
    loss, lse = xent.loss(P, x, target)
    dx, _ = xent.backward(P, x, target, lse, grad)
    for t in range(m):
        z = wv * X[t]
        ref = torch.logsumexp(z, 0)
        # products of 4-bit significands are exact; a thread joins up to 8192 of the
        # partial sums of 256 entries one after another
        tol = 2.0 ** -17 + 16 * 8192 ** 0.5 * 2.0 ** -24 + 2.0 ** -22 * abs(float(ref))
        assert abs(float(lse[t]) - float(ref)) <= tol
        assert abs(float(loss[t]) - float(ref - z[target[t]])) <= tol
        p = torch.exp(z - ref)
        G = p.clone()
        G[target[t]] -= 1.0
        terms = G * wv * float(grad[t])
        # p is off by the exponential and by lse; dz's rounding is the same for all
        # entries of one code, so it adds up in full
        part = (2.0 ** -17 + tol) * float((p * wv).abs().sum()) * abs(float(grad[t]))
        spread = (H + n ** 0.5 * 2.0 ** -24) * float(terms.abs().sum()) + 2.0 ** -126 * n
        want = float(terms.sum())
        assert abs(float(dx[t, 0]) - want) <= spread + part + H * abs(want), t


@pytest.mark.parametrize("m", [3, 70])
@pytest.mark.parametrize("head", ["packed", "f8"])
def test_longest_k(m, head):
    room(32)
    n, n_vocab, k = 256, 200, 1 << 21
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(n, k, generator=g, device="cuda") * 2.0 ** -11).bfloat16()
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    target = torch.randint(0, n_vocab, (m,), generator=g, device="cuda")
    grad = torch.randn(m, generator=g, device="cuda")
    if head == "packed":
        P = hb.pack(w, (torch.arange(n // 64 * (k // 256)) % 3 == 0).view(n // 64, -1).to(torch.uint8).numpy(), 64, 256)
        xv, wv = x.double(), hb.unpack(P).double()[:n_vocab]
    else:
        P = f8.pack(w)
        xv = f8.unpack(f8.quant(x), out_dtype=torch.float32).double()
        wv = f8.unpack(P).double()[:n_vocab]
    loss, lse = xent.loss(P, x, target, n_vocab=n_vocab)
    dx, dw = xent.backward(P, x, target, lse, grad, n_vocab=n_vocab, need_dw=head == "packed")
    z = xv @ wv.t()
    ez = 16 * k ** 0.5 * 2.0 ** -23 * ((xv * xv) @ (wv * wv).t()).sqrt().amax(1)
    ref = torch.logsumexp(z, 1)
    tol = 2 * ez + 2.0 ** -17 + 2.0 ** -22 * ref.abs()
    assert bool(((lse - ref).abs() <= tol).all())
    assert bool(((loss - (ref - z.gather(1, target[:, None])[:, 0])).abs() <= tol).all())
    p = torch.exp(z - ref[:, None])
    G = p.scatter_add(1, target[:, None], torch.full((m, 1), -1.0, dtype=torch.float64, device="cuda"))
    ag = grad.double().abs()[:, None]
    eg = (G.abs() * (H + 256 * 2.0 ** -23) + p * (ez + 2.0 ** -17)[:, None]) * ag
    want = (G * grad.double()[:, None]) @ wv
    assert bool(((dx - want).abs() <= eg @ wv.abs() + H * want.abs() + 2.0 ** -126).all())
    if dw is not None:
        want = (G * grad.double()[:, None]).t() @ xv
        assert bool(((dw[:n_vocab] - want).abs() <= eg.t() @ xv.abs() + H * want.abs() + 2.0 ** -126).all())
        assert bool((dw[n_vocab:] == 0).all())
