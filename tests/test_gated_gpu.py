"""The gated projection and its gradients on the GPU against the float64 oracle.

Forward.  G and U are fp32 sums of exact products: off by at most k * 2^-23 * S
(S = sum |x w|) each.  act has a slope of at most 1.2 everywhere, and its fp32
evaluation is off by at most (|g|^3 + |g| + 8) * 2^-23 * |g|: a few roundings, and
the rounding of the exponential's argument (at most 3 * 2 c (|g| + 0.045 |g|^3) *
2^-24 relative).  H = act(G) U is then rounded to 16 bits, half a step.

Backward, from the fp32 G and U that the call is given: dG and dU are rounded to
16 bits (half a step; fp16 holds them scaled, off by 2^-38 of the largest one at
least), the sums are fp32 (a rounding of 2^-23 of the absolute sum for each term)
and each output is rounded by half a step."""
import numpy as np
import pytest
import torch

import oracle
from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated, q4
from oracle import gated_oracle as go
from oracle import q4_oracle as qo

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"bf16": 0.0, "f16": 2.0 ** -25}


def normal(seed, rows, cols, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * scale).to(DT[dtype]).cuda()


def as64(t):
    return t.detach().cpu().double().numpy()


def packed(seed, n, k, dtype, sparse, b1=64, b2=64, meta="idx2", scale=None):
    """A packed weight and, in float64, what its streams stand for."""
    w = normal(seed, n, k, dtype, scale or k ** -0.5)
    tiles = (np.random.default_rng(seed).random((n // b1, k // b2)) < sparse).astype(np.uint8)
    P = hb.pack(w, tiles, b1, b2, meta)
    bits = oracle.prune(hb.tensor_to_bits(w), tiles, b1, b2, **({"meta": meta} if meta == "mask8" else {}))
    return P, as64(hb.bits_to_tensor(bits, dtype, "cpu"))


def weights(kind, seed, n, k, dtype, sparse=0.5, **more):
    if kind == "packed":
        return packed(seed, n, k, dtype, sparse, **more) + packed(seed + 1, n, k, dtype, sparse, **more)
    a, b = (normal(seed + i, n, k, dtype, k ** -0.5) for i in range(2))
    return q4.pack(a), qo.values(*qo.quantise(as64(a))), q4.pack(b), qo.values(*qo.quantise(as64(b)))


def close(got, ref, tol):
    err = np.abs(as64(got) - ref)
    bad = np.argwhere(~(err <= tol))
    assert bad.size == 0, (len(bad), bad[:4].tolist(), float(np.nanmax(err - tol)), float(np.abs(ref).max()))


def act_error(g):
    return (np.abs(g) ** 3 + np.abs(g) + 8.0) * 2.0 ** -23 * np.abs(g)


def check_forward(G, wg, U, wu, x, dtype, act, save=False):
    k = x.shape[1]
    xv = as64(x)
    g, u, h = go.forward(xv, wg, wu, act)
    eg = k * 2.0 ** -23 * (np.abs(xv) @ np.abs(wg).T)
    eu = k * 2.0 ** -23 * (np.abs(xv) @ np.abs(wu).T)
    a = go.act(g, act)[0]
    ea = 1.2 * eg + act_error(np.abs(g) + eg)
    tol = (np.abs(a) + ea) * eu + ea * np.abs(u)
    out = gated.forward(G, U, x, act=act, save=save)
    close(out[0] if save else out, h, tol + HALF[dtype] * (np.abs(h) + tol) + LEAST[dtype])
    if save:
        assert out[1].dtype == out[2].dtype == torch.float32
        close(out[1], g, eg)
        close(out[2], u, eu)
    return out


def check_backward(G, wg, U, wu, x, g, u, dh, dtype, act, got):
    """`got` = (dx, dw_gate, dw_up), None where not asked for."""
    xv, gv, uv, dv = as64(x), as64(g), as64(u), as64(dh)
    m, n = gv.shape
    dg, du = go.gradients(gv, uv, dv, act)
    a, slope = go.act(gv, act)
    # the slope's own error: as act's, with one power of g more from g act''
    es = (np.abs(gv) ** 3 + np.abs(gv) + 8.0) * 2.0 ** -22 * (1.0 + np.abs(gv))
    eg = np.abs(dv * uv) * (es + 2.0 ** -22 * np.abs(slope))
    eu = np.abs(dv) * (act_error(gv) + 2.0 ** -23 * np.abs(a))
    top = 0.0
    if dtype == "f16":
        both = np.concatenate([np.abs(dg).ravel(), np.abs(du).ravel()])
        both = both[np.isfinite(both)]
        top = float(both.max()) * 2.0 ** -37 if both.size else 0.0
    eg = eg + HALF[dtype] * (np.abs(dg) + eg) + top
    eu = eu + HALF[dtype] * (np.abs(du) + eu) + top
    ag, au = np.abs(dg) + eg, np.abs(du) + eu

    def rounded(ref, tol):
        return tol + HALF[dtype] * (np.abs(ref) + tol) + LEAST[dtype]

    dx, dwg, dwu = got
    if dx is not None:
        ref = dg @ wg + du @ wu
        s = ag @ np.abs(wg) + au @ np.abs(wu)
        close(dx, ref, rounded(ref, eg @ np.abs(wg) + eu @ np.abs(wu) + 2 * n * 2.0 ** -23 * s))
    for dw, d, e, ad in ((dwg, dg, eg, ag), (dwu, du, eu, au)):
        if dw is not None:
            ref = d.T @ xv
            close(dw, ref, rounded(ref, e.T @ np.abs(xv) + m * 2.0 ** -23 * (ad.T @ np.abs(xv))))


# ----------------------------------------------------------------- forward --

@pytest.mark.parametrize("m", [1, 3, 4, 5, 16, 17, 64, 65, 130, 300])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu"), ("bf16", "gelu_tanh")])
@pytest.mark.parametrize("n,k", [(64, 64), (192, 320), (320, 1024)])
def test_forward_packed(m, dtype, act, n, k):
    check_forward(*weights("packed", n + k, n, k, dtype), normal(m, m, k, dtype), dtype, act, save=m % 2 == 1)


@pytest.mark.parametrize("m", [2, 20, 140])
@pytest.mark.parametrize("b1,b2,meta", [(128, 64, "idx2"), (64, 256, "mask4"), (256, 128, "mask8")])
@pytest.mark.parametrize("sparse", [0.0, 0.5, 1.0])
def test_forward_tiles(m, b1, b2, meta, sparse):
    ws = weights("packed", 5, 512, 512, "bf16", sparse, b1=b1, b2=b2, meta=meta)
    check_forward(*ws, normal(6, m, 512, "bf16"), "bf16", "silu", save=True)


@pytest.mark.parametrize("m", [1, 2, 5, 9, 16, 17, 40, 65, 130, 300])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu"), ("f16", "gelu_tanh")])
@pytest.mark.parametrize("n,k", [(64, 64), (129, 300), (300, 1501), (1, 2100)])
def test_forward_4bit(m, dtype, act, n, k):
    check_forward(*weights("4bit", n + k, n, k, dtype), normal(m, m, k, dtype), dtype, act)


@pytest.mark.parametrize("kind", ["packed", "4bit"])
@pytest.mark.parametrize("m", [1, 16, 200])
def test_forward_large_arguments(kind, m):
    """Gates up to a few hundred: act is 0 or its argument."""
    n, k = 128, 256
    for act in gated.ACTS:
        G, wg, U, wu = weights(kind, 3, n, k, "bf16")
        x = normal(4, m, k, "bf16", 60.0)
        y = as64(gated.forward(G, U, x, act=act))
        g, u, h = go.forward(as64(x), wg, wu, act)
        assert np.isfinite(y).all()
        far = np.abs(g) > 40
        assert far.any()
        eg = k * 2.0 ** -23 * (np.abs(as64(x)) @ np.abs(wg).T)
        eu = k * 2.0 ** -23 * (np.abs(as64(x)) @ np.abs(wu).T)
        tol = 2.0 ** -8 * np.abs(h) + 2 * (eg * np.abs(u) + eu * np.abs(g)) + 1e-9
        assert (np.abs(y - h) <= tol)[far].all()


@pytest.mark.parametrize("kind", ["packed", "4bit"])
@pytest.mark.parametrize("m", [1, 3, 16, 30, 100, 300])
def test_rows_stay_apart(kind, m):
    """A NaN token makes its own outputs NaN only; strides and what lies between
    the rows are left alone."""
    n, k = 128, 256
    G, wg, U, wu = weights(kind, 8, n, k, "bf16")
    x = torch.full((m + 3, k + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:m, :k] = normal(9, m, k, "bf16")
    base = torch.full((m + 1, n + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    h = gated.forward(G, U, x[:m, :k], out=base[:m, 2:n + 2])
    ref = check_forward(G, wg, U, wu, x[:m, :k].contiguous(), "bf16", "silu")
    assert torch.equal(h, ref)
    base[:m, 2:n + 2] = 7.0
    assert bool((base == 7.0).all())
    x[m - 1, 5] = float("inf")
    y = gated.forward(G, U, x[:m, :k])
    assert torch.equal(y[:m - 1], ref[:m - 1]) and not bool(torch.isfinite(y[m - 1]).all())


# ---------------------------------------------------------------- backward --

@pytest.mark.parametrize("m", [1, 5, 16, 17, 64, 65, 129, 260, 300])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu"), ("f16", "silu"), ("bf16", "gelu_tanh")])
@pytest.mark.parametrize("n,k", [(64, 64), (192, 320), (1024, 256)])
def test_backward(m, dtype, act, n, k):
    G, wg, U, wu = weights("packed", n + k, n, k, dtype)
    x, dh = normal(m, m, k, dtype), normal(m + 1, m, n, dtype, 0.1)
    _, g, u = gated.forward(G, U, x, act=act, save=True)
    got = gated.backward(G, U, x, g, u, dh, act=act, need_dw=True)
    check_backward(G, wg, U, wu, x, g, u, dh, dtype, act, got)
    dx = gated.backward(G, U, x, g, u, dh, act=act)
    assert dx[1] is None and dx[2] is None and torch.equal(dx[0], got[0])
    dw = gated.backward(G, U, x, g, u, dh, act=act, need_dx=False, need_dw=True)
    assert dw[0] is None and torch.equal(dw[1], got[1]) and torch.equal(dw[2], got[2])


@pytest.mark.parametrize("m", [20, 140])
@pytest.mark.parametrize("b1,b2,meta", [(128, 64, "idx2"), (64, 256, "mask4"), (256, 128, "mask8")])
@pytest.mark.parametrize("sparse", [0.0, 0.5, 1.0])
def test_backward_tiles(m, b1, b2, meta, sparse):
    G, wg, U, wu = weights("packed", 5, 512, 512, "bf16", sparse, b1=b1, b2=b2, meta=meta)
    x, dh = normal(6, m, 512, "bf16"), normal(7, m, 512, "bf16")
    _, g, u = gated.forward(G, U, x, save=True)
    check_backward(G, wg, U, wu, x, g, u, dh, "bf16", "silu", gated.backward(G, U, x, g, u, dh, need_dw=True))


@pytest.mark.parametrize("m,n,k", [(1, 8192, 512), (40, 4096, 1024), (600, 512, 512)])
def test_backward_larger(m, n, k):
    G, wg, U, wu = weights("packed", 15, n, k, "bf16", b1=128, b2=128)
    x, dh = normal(16, m, k, "bf16"), normal(17, m, n, "bf16")
    _, g, u = gated.forward(G, U, x, save=True)
    check_backward(G, wg, U, wu, x, g, u, dh, "bf16", "silu", gated.backward(G, U, x, g, u, dh, need_dw=True))


@pytest.mark.parametrize("scale", [2.0 ** -18, 2.0 ** 9])
def test_backward_f16_range(scale):
    """Gradients that fp16 alone would flush to zero, or overflow before the
    sums bring them back."""
    m, n, k = 80, 128, 192
    G, wg, U, wu = weights("packed", 25, n, k, "f16", scale=2.0 ** -9 if scale > 1 else None)
    x = normal(26, m, k, "f16")
    g, u = normal(27, m, n, "f16", 4.0).float(), normal(28, m, n, "f16", 60.0).float()
    dh = normal(29, m, n, "f16", scale)
    got = gated.backward(G, U, x * 0.001 if scale > 1 else x, g, u, dh, need_dw=True)
    xs = x * 0.001 if scale > 1 else x
    assert all(bool(torch.isfinite(t).all()) for t in got)
    check_backward(G, wg, U, wu, xs, g, u, dh, "f16", "silu", got)


def test_backward_zero_and_nan_gradients():
    m, n, k = 70, 128, 128
    for dtype in DT:
        G, wg, U, wu = weights("packed", 35, n, k, dtype)
        x = normal(36, m, k, dtype)
        h, g, u = gated.forward(G, U, x, save=True)
        zero = gated.backward(G, U, x, g, u, torch.zeros_like(h), need_dw=True)
        assert all(bool((t == 0).all()) for t in zero)
        dh = normal(37, m, n, dtype)
        want = gated.backward(G, U, x, g, u, dh, need_dw=True)
        dh[3, 5] = float("nan")
        dx, dwg, dwu = gated.backward(G, U, x, g, u, dh, need_dw=True)
        rows = torch.arange(m, device="cuda") != 3
        cols = torch.arange(n, device="cuda") != 5
        assert bool(dx[3].isnan().all()) and bool(dwg[5].isnan().all()) and bool(dwu[5].isnan().all())
        assert torch.equal(dx[rows], want[0][rows])
        assert torch.equal(dwg[cols], want[1][cols]) and torch.equal(dwu[cols], want[2][cols])


@pytest.mark.parametrize("m", [7, 100])
def test_backward_strides(m):
    n, k = 128, 192
    G, wg, U, wu = weights("packed", 45, n, k, "bf16")
    x = normal(46, m, k, "bf16")
    _, g, u = gated.forward(G, U, x, save=True)
    dh = normal(47, m, n, "bf16")
    want = gated.backward(G, U, x, g, u, dh, need_dw=True)

    def wide(t, pad, off):
        big = torch.full((t.shape[0] + 1, t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        big[:t.shape[0], off:off + t.shape[1]] = t
        return big, big[:t.shape[0], off:off + t.shape[1]]
    outs = [wide(torch.zeros_like(t), p, o) for t, p, o in zip(want, (3, 5, 8), (1, 0, 3))]
    got = gated.backward(G, U, wide(x, 8, 0)[1], wide(g, 3, 1)[1], wide(u, 2, 2)[1], wide(dh, 1, 0)[1],
                         dx=outs[0][1], dw_gate=outs[1][1], dw_up=outs[2][1])
    for a, b, (big, view) in zip(got, want, outs):
        assert a.data_ptr() == view.data_ptr() and torch.equal(a, b)
        view.fill_(float("nan"))
        assert bool(big.isnan().all())


def test_empty_batch():
    G, _, U, _ = weights("packed", 55, 64, 64, "bf16")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    h, g, u = gated.forward(G, U, x, save=True)
    assert h.shape == g.shape == u.shape == (0, 64)
    dx, dwg, dwu = gated.backward(G, U, x, g, u, h, need_dw=True)
    assert dx.shape == (0, 64) and bool((dwg == 0).all()) and bool((dwu == 0).all())
    A, _, B, _ = weights("4bit", 56, 5, 70, "bf16")
    assert gated.forward(A, B, torch.empty(0, 70, dtype=torch.bfloat16, device="cuda")).shape == (0, 5)


# ------------------------------------------------------------------ as used --

@pytest.mark.parametrize("m", [2, 40, 300])
def test_graph_capture(m):
    """Forward and backward captured once and replayed on new inputs, eager work
    in between."""
    n, k = 256, 320
    for dtype in DT:
        G, _, U, _ = weights("packed", 65, n, k, dtype)
        x, dh = normal(66, m, k, dtype), normal(67, m, n, dtype)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            h, g, u = gated.forward(G, U, x, save=True)
            gated.backward(G, U, x, g, u, dh, need_dw=True)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h, g, u = gated.forward(G, U, x, save=True)
            grads = gated.backward(G, U, x, g, u, dh, need_dw=True)
        for seed in range(3):
            x.copy_(normal(70 + seed, m, k, dtype))
            dh.copy_(normal(80 + seed, m, n, dtype, 10.0 ** -seed))
            graph.replay()
            torch.cuda.synchronize()
            want = gated.forward(G, U, x, save=True)
            again = gated.backward(G, U, x, want[1], want[2], dh, need_dw=True)
            for a, b in zip((h, g, u) + tuple(grads), want + tuple(again)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("m", [3, 30, 200])
def test_two_streams_at_once(m):
    n, k = 256, 512
    jobs = []
    for i in range(2):
        G, _, U, _ = weights("packed" if i else "4bit", 90 + i, n, k, "bf16")
        x = normal(95 + i, m, k, "bf16")
        jobs.append((G, U, x, gated.forward(G, U, x)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(5):
        for s, (G, U, x, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(gated.forward(G, U, x))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, jobs[i % 2][3])


def test_workspace_of_the_caller():
    n, k, m = 256, 320, 300
    G, _, U, _ = weights("packed", 101, n, k, "f16")
    x, dh = normal(102, m, k, "f16"), normal(103, m, n, "f16")
    h, g, u = gated.forward(G, U, x, save=True)
    grads = gated.backward(G, U, x, g, u, dh, need_dw=True)
    need = max(gated.workspace_bytes(G, U, m), gated.workspace_bytes(G, U, m, dx=True, dw=True))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(gated.forward(G, U, x, workspace=ws), h)
    for a, b in zip(gated.backward(G, U, x, g, u, dh, need_dw=True, workspace=ws), grads):
        assert torch.equal(a, b)
    with pytest.raises(hb.HybError):
        gated.backward(G, U, x, g, u, dh, need_dw=True, workspace=ws[:1024])


def test_more_than_2_31_outputs():
    """G, U, H and the gradients' panels lie beyond 2^31 elements; only the last
    tokens have a gradient."""
    m, n, k, last = 160000, 14336, 64, slice(159700, 160000)
    G, wg, U, wu = weights("packed", 7, n, k, "bf16")
    x = normal(8, m, k, "bf16")
    h, g, u = gated.forward(G, U, x, save=True)
    xv = as64(x[last])
    for got, w in ((g, wg), (u, wu)):
        close(got[last], xv @ w.T, k * 2.0 ** -23 * (np.abs(xv) @ np.abs(w).T))
    a = go.act(as64(g[last]), "silu")[0]
    ref = a * as64(u[last])
    close(h[last], ref, (2.0 ** -8 + 2.0 ** -20) * np.abs(ref) + act_error(as64(g[last])) * np.abs(as64(u[last])))
    dh = torch.zeros_like(h)
    dh[last] = normal(9, 300, n, "bf16")
    dx, dwg, dwu = gated.backward(G, U, x, g, u, dh, need_dw=True)
    assert not dx[:159700].any()
    check_backward(G, wg, U, wu, x[last], g[last], u[last], dh[last], "bf16", "silu", (dx[last], dwg, dwu))
