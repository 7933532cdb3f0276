"""A training step of a gated projection under a vocabulary projection, and its
weights served in four bits: forward, loss, gradients, clipping, update, 4-bit
packing, decode.  Each operator is checked against float64 on what the operator
before it gave, with the bounds of its own tests; the whole is then captured once
and replayed."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import clip, gated, q4, xent
from oracle import q4_oracle as qo
from test_clip_gpu import check as check_clip
from test_gated_gpu import DT, as64, check_backward, check_forward, normal, packed
from test_xent_gpu import bounds, operands, within

pytestmark = pytest.mark.gpu

VOCAB, FFN, HIDDEN = 500, 576, 320  # the vocabulary projection has 512 rows


def model(dtype, seed=1):
    G, wg = packed(seed, FFN, HIDDEN, dtype, 0.5)
    U, wu = packed(seed + 1, FFN, HIDDEN, dtype, 0.3)
    V, _ = packed(seed + 2, 512, FFN, dtype, 0.5)
    return G, wg, U, wu, V


def targets(seed, m):
    t = torch.from_numpy(np.random.default_rng(seed).integers(0, VOCAB, m))
    t[1::5] = -100
    return t.cuda()


def step(G, U, V, x, target, grad):
    """One training step's tensors."""
    h, g, u = gated.forward(G, U, x, save=True)
    loss, lse = xent.loss(V, h, target, n_vocab=VOCAB)
    dh, dv = xent.backward(V, h, target, lse, grad, n_vocab=VOCAB, need_dw=True)
    dx, dwg, dwu = gated.backward(G, U, x, g, u, dh, need_dw=True)
    outs = [torch.empty_like(t) for t in (dv, dwg, dwu)]
    norm = clip.clip([dv, dwg, dwu], 0.01, outs=outs)
    return h, g, u, loss, lse, dh, dv, dx, dwg, dwu, norm, *outs


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 6, 100, 301])
def test_step_and_serving(m, dtype):
    G, wg, U, wu, V = model(dtype)
    x, target = normal(5, m, HIDDEN, dtype), targets(6, m)
    grad = torch.full((m,), 1.0 / m, device="cuda")
    h, g, u, loss, lse, dh, dv, dx, dwg, dwu, norm, *clipped = step(G, U, V, x, target, grad)

    again = check_forward(G, wg, U, wu, x, dtype, "silu", save=True)
    assert all(torch.equal(a, b) for a, b in zip(again, (h, g, u)))
    hv, vv = operands(V, None, h)
    want, tol = bounds(hv, vv, h, target, grad, VOCAB, FFN)
    for name, got, w, t in zip(("loss", "lse", "dh", "dv"), (loss, lse, dh, dv), want, tol):
        within(name, got, w, t)
    assert not dh[target == -100].any() and not dx[target == -100].any()
    check_backward(G, wg, U, wu, x, g, u, dh, dtype, "silu", (dx, dwg, dwu))
    check_clip([dv, dwg, dwu], 0.01, clipped, norm)

    # the updated weights, in four bits
    new = [torch.from_numpy(w).to(DT[dtype]).cuda() - d for w, d in zip((wg, wu), clipped[1:])]
    Q = [q4.pack(w) for w in new]
    values = [qo.values(*qo.quantise(as64(w))) for w in new]
    for q, v in zip(Q, values):
        assert np.array_equal(as64(q4.unpack(q, out_dtype=torch.float32)), v)
    for rows in (x, x[:1]):
        check_forward(Q[0], values[0], Q[1], values[1], rows, dtype, "silu")
    W = q4.pack(torch.from_numpy(vv).to(DT[dtype]).cuda())
    dense = qo.values(*qo.quantise(vv))
    y = q4.gemm(W, h, out_dtype=torch.float32)
    err = np.abs(as64(y) - hv @ dense.T)
    assert (err <= FFN * 2.0 ** -23 * (np.abs(hv) @ np.abs(dense).T) + 2.0 ** -126).all()


@pytest.mark.parametrize("m", [3, 100, 301])
def test_step_captured(m):
    G, _, U, _, V = model("bf16")
    x, target = normal(5, m, HIDDEN, "bf16"), targets(6, m)
    grad = torch.full((m,), 1.0 / m, device="cuda")

    def run():
        out = step(G, U, V, x, target, grad)
        Q = q4.pack(out[-1]), q4.pack(out[-2])
        return *out, Q[0].codes, Q[0].scales, Q[1].codes, Q[1].scales, gated.forward(*Q, x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in range(3):
        x.copy_(normal(20 + seed, m, HIDDEN, "bf16"))
        target.copy_(targets(30 + seed, m))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, run()):
            assert torch.equal(a, b)
