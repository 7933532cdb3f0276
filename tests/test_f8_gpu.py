"""8-bit block-scaled matrices on the GPU against the float64 oracle.

Codes, scales and values read back have to match bit for bit.  A product's
terms are exact (4-bit by 4-bit significands and powers of two), so its error
is that of fp32 summation: at most k roundings or truncations of a partial sum
that is at most S = sum |x w|, that is k * 2^-23 * S, and for a 16-bit output
half a step (2^-8 or 2^-11) of the result on top.  16-bit outputs may come from
the 8-bit matrix instruction: 2^-11 of each step's largest product more
(bounded by the product of the two rows' largest elements)."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import f8
from oracle import f8_oracle as fo

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def normal(seed, rows, k, dtype, scale=1.0, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, k, generator=g) * scale).to(DT[dtype]).to(dev)


def as64(t):
    return t.detach().cpu().double().numpy()


def check_quantised(a, kind):
    block = 128 if kind == f8.WEIGHT else 1
    Q = f8.pack(a) if kind == f8.WEIGHT else f8.quant(a)
    codes, exps = fo.quantise(as64(a), block)
    cb, sb = fo.buffers(codes, exps)
    assert np.array_equal(Q.scales.cpu().numpy(), sb)
    got = Q.codes.cpu().numpy()
    off = np.flatnonzero(got != cb)
    assert off.size == 0, (off.size, off[:8].tolist(), got[off[:8]].tolist(), cb[off[:8]].tolist())
    want = fo.values(codes, exps)
    for dt in DT.values():
        got = as64(f8.unpack(Q, out_dtype=dt))
        ref = torch.from_numpy(want).to(dt).double().numpy()
        assert np.array_equal(got, ref, equal_nan=True), dt
    # exact in the type quantised, but where a value near the type's largest
    # rounds up past it (bf16: 255 / 256 * 2^128 has the quotient 255, whose
    # nearest code is 256: 2^128)
    inside = ~(np.abs(want) > torch.finfo(a.dtype).max)
    assert np.array_equal(as64(f8.unpack(Q))[inside], want[inside], equal_nan=True)
    return Q, want


@pytest.mark.parametrize("kind", [f8.WEIGHT, f8.ROWS])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 128), (16, 512), (17, 127), (127, 640), (129, 300), (300, 1501), (1, 4096)])
def test_quantise(kind, dtype, rows, k):
    check_quantised(normal(rows * 7 + k, rows, k, dtype, 0.3), kind)


@pytest.mark.parametrize("kind", [f8.WEIGHT, f8.ROWS])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantise_special_values(kind, dtype):
    a = normal(5, 260, 700, dtype)
    a[3] = 0.0                                       # a row, and a block, of zeros
    a[128:256, 128:256] = 0.0
    a[5, 7], a[6, 200], a[259, 699] = float("inf"), float("-inf"), float("nan")
    a[130, 300:428] = float("nan")                   # nothing finite in a row's block
    a[7] *= 2.0 ** -20 if dtype == "f16" else 2.0 ** -130   # subnormal in every type
    a[8] *= 2.0 ** 10
    a[9, :128] = 448.0
    a[10, :128] = 448.0 * 2
    a[11, 5] = torch.finfo(DT[dtype]).max
    a[12, 0] = torch.finfo(DT[dtype]).smallest_normal
    a[13, 0] = -0.0
    check_quantised(a, kind)


@pytest.mark.parametrize("kind", [f8.WEIGHT, f8.ROWS])
def test_quantise_every_halfway_point(kind):
    grid = fo.e4m3_table()[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([mid, -mid, grid, -grid]).astype(np.float32)
    v = np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(448)) * (np.abs(v) < 448)])
    a = torch.from_numpy(np.resize(v, (16, 128 * 7)).astype(np.float32)).cuda()
    a[:, ::128] = 448.0                              # every block's scale is 1
    check_quantised(a, kind)


@pytest.mark.parametrize("offset,pitch", [(0, 712), (1, 713), (8, 720), (3, 704)])
def test_quantise_strides(offset, pitch):
    base = normal(9, 40, pitch + 16, "bf16").flatten()
    a = torch.as_strided(base, (37, 700), (pitch, 1), offset)
    for kind in (f8.WEIGHT, f8.ROWS):
        Q, want = check_quantised(a, kind)
        out = torch.full((40 * (pitch + 16),), 7.0, dtype=torch.bfloat16, device="cuda")
        view = torch.as_strided(out, (37, 700), (pitch, 1), offset)
        f8.unpack(Q, out=view)
        assert np.array_equal(as64(view), want)
        rest = torch.ones_like(out, dtype=torch.bool)
        torch.as_strided(rest, (37, 700), (pitch, 1), offset).fill_(False)
        assert bool((out[rest] == 7.0).all())        # nothing between or behind the rows


def step_tops(a):
    return np.abs(np.pad(a, ((0, 0), (0, -a.shape[1] % 128)))).reshape(a.shape[0], -1, 128).max(2)


def reference(x, w):
    """The product in float64, and the two sums of its error bound."""
    xv = fo.values(*fo.quantise(as64(x), 1))
    wv = fo.values(*fo.quantise(as64(w), 128))
    return xv @ wv.T, (np.abs(xv) @ np.abs(wv).T, step_tops(xv) @ step_tops(wv).T)


def check_product(y, ref, s, k):
    tol = k * 2.0 ** -23 * s[0] + HALF[y.dtype] * np.abs(ref) + (2.0 ** -25 if y.dtype == torch.float16 else 0.0)
    if y.dtype != torch.float32:
        tol += 2.0 ** -11 * s[1]
    err = np.abs(as64(y) - ref)
    print("worst error over bound", float(np.max(err / np.maximum(tol, 1e-300))))
    assert np.all(err <= tol), (float(np.max(err - tol)), np.argwhere(err > tol)[:4].tolist(), int((err > tol).sum()))


@pytest.mark.parametrize("m", [1, 2, 5, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 200, 256, 300])
@pytest.mark.parametrize("n,k", [(300, 1501), (128, 128), (1000, 640), (17, 5000)])
def test_product(m, n, k):
    x, w = normal(m, m, k, "bf16"), normal(n + k, n, k, "bf16", 0.05)
    x[:, 0] *= 50.0
    ref, s = reference(x, w)
    check_product(f8.gemm(f8.pack(w), x), ref, s, k)


@pytest.mark.parametrize("m,n,k,dtype,out", [
    (1, 14336, 256, "bf16", "f32"), (16, 4096, 4096, "f16", "f16"), (1, 1, 1, "f32", "f32"), (3, 2, 129, "f32", "bf16"),
    (4096, 4096, 300, "bf16", "bf16"), (4000, 5000, 1030, "f16", "f16"), (2048, 8300, 128, "bf16", "f32"),
    (700, 1500, 5000, "bf16", "f32"), (256, 1024, 8192, "bf16", "bf16"), (512, 640, 28672, "bf16", "f32"),
    (80, 3000, 28672, "bf16", "f32"), (1, 16, 28672, "bf16", "f32"), (33, 130, 1 << 18, "bf16", "f32"),
])
def test_product_shapes_and_types(m, n, k, dtype, out):
    x, w = normal(m, m, k, dtype), normal(n + k, n, k, dtype, 0.05)
    ref, s = reference(x, w)
    check_product(f8.gemm(f8.pack(w), x, out_dtype=DT[out]), ref, s, k)


def test_product_exact_integers():
    """Small integers: every sum is exact, so the result is the product's."""
    g = torch.Generator().manual_seed(1)
    for m, n, k in [(1, 200, 700), (40, 200, 700), (300, 500, 700), (2100, 8200, 384)]:
        x = torch.randint(-8, 9, (m, k), generator=g).to(torch.bfloat16)
        w = torch.randint(-8, 9, (n, k), generator=g).to(torch.bfloat16)
        y = f8.gemm(f8.pack(w.cuda()), x.cuda())
        assert torch.equal(y.cpu(), x.float() @ w.float().t()), (m, n, k)


def test_product_scales_vary():
    """Each block its own scale, over 40 binades: a scale taken from a
    neighbouring row, step or block would be off by powers of two."""
    for m, n, k in [(1, 300, 1100), (20, 300, 1100), (150, 400, 1100), (2100, 8200, 900)]:
        x, w = normal(1, m, k, "f32"), normal(2, n, k, "f32")
        g = torch.Generator().manual_seed(3)
        sx = torch.randint(-10, 11, (m, -(-k // 128)), generator=g).float().exp2()
        sw = torch.randint(-10, 11, (-(-n // 128), -(-k // 128)), generator=g).float().exp2()
        x *= sx.repeat_interleave(128, 1)[:, :k].cuda()
        w *= sw.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k].cuda()
        ref, s = reference(x, w)
        check_product(f8.gemm(f8.pack(w), x), ref, s, k)


@pytest.mark.parametrize("m", [1, 20, 130])
def test_product_output_views_and_reused_activations(m):
    n, k = 210, 900
    x, w = normal(m, m, k, "bf16"), normal(3, n, k, "bf16", 0.05)
    ref, s = reference(x, w)
    Q, X = f8.pack(w), f8.quant(x)
    for dt in DT.values():
        for pitch, offset in [(n, 0), (n + 5, 3), (n + 6, 4)]:
            buf = torch.full((m * pitch + 64,), 9.0, dtype=dt, device="cuda")
            view = torch.as_strided(buf, (m, n), (pitch, 1), offset)
            f8.gemm(Q, X, out=view)
            check_product(view, ref, s, k)
            rest = torch.ones_like(buf, dtype=torch.bool)
            torch.as_strided(rest, (m, n), (pitch, 1), offset).fill_(False)
            assert bool((buf[rest] == 9.0).all())
    # the same activations through a second matrix, into reused buffers
    w2 = normal(4, n, k, "bf16", 0.05)
    f8.pack(w2, out=Q)
    ref2, s2 = reference(x, w2)
    check_product(f8.gemm(Q, X), ref2, s2, k)


@pytest.mark.parametrize("m", [2, 40, 140, 2100])
def test_product_not_finite(m):
    """A token or weight row with a NaN or an infinity is NaN where it is
    read and touches no other output."""
    n, k = 300 if m < 2000 else 8200, 640
    x, w = normal(m, m, k, "bf16"), normal(3, n, k, "bf16", 0.05)
    clean = f8.gemm(f8.pack(w), x)
    x[1, 3], w[7, 300] = float("nan"), float("inf")
    y = f8.gemm(f8.pack(w), x)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[1], bad[:, 7] = True, True
    assert bool(y[bad].isnan().all()) and bool(y[~bad].isfinite().all())
    same = ~bad
    same[:, :128] = False        # block of the infinity: its scale may differ
    assert torch.equal(y[same], clean[same])


@pytest.mark.parametrize("m", [0, 1, 3])
def test_empty(m):
    w, x = torch.zeros(20, 0, dtype=torch.bfloat16, device="cuda"), torch.zeros(m, 0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((m, 20), 5.0, device="cuda")
    f8.gemm(f8.pack(w), x, out=out)
    assert bool((out == 0).all())
    w = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    assert f8.gemm(f8.pack(w), torch.zeros(m, 64, device="cuda")).shape == (m, 0)
    assert f8.unpack(f8.quant(torch.zeros(m, 64, device="cuda"))).shape == (m, 64)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_graph_replays(m):
    n, k = 1024, 8192
    x, w = normal(1, m, k, "bf16"), normal(2, n, k, "bf16", 0.05)
    Q = f8.pack(w)
    f8.gemm(Q, x)
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    x2 = normal(7, m, k, "bf16")
    with torch.cuda.graph(graph):
        y = f8.gemm(Q, x)
    with torch.cuda.graph(other):
        y2 = f8.gemm(Q, x2)
    for seed in (3, 4, 5):
        x.copy_(normal(seed, m, k, "bf16"))
        x2.copy_(normal(seed + 10, m, k, "bf16"))
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, f8.gemm(Q, x)) and torch.equal(y2, f8.gemm(Q, x2))
        torch.cuda.synchronize()


def test_two_streams():
    n, k = 1024, 8192
    w = normal(2, n, k, "bf16", 0.05)
    Q = f8.pack(w)
    xs = [normal(i, m, k, "bf16") for i, m in enumerate((300, 300, 40, 1))]
    want = [f8.gemm(Q, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(f8.gemm(Q, xs[i]))
    torch.cuda.synchronize()
    for i, w_ in enumerate(want):
        assert all(torch.equal(g, w_) for g in got[i]), i


@pytest.mark.parametrize("m", [1, 2, 3, 4, 16, 70, 300, 2100])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_one_call_is_quantise_then_product(m, dtype):
    n, k = 1100, 3000
    x, w = normal(m, m, k, dtype), normal(3, n, k, dtype, 0.05)
    Q = f8.pack(w)
    for dt in (torch.float32, torch.bfloat16):
        want = f8.gemm(Q, f8.quant(x), out_dtype=dt)
        assert torch.equal(f8.gemm(Q, x, out_dtype=dt), want)
        ws = torch.full((f8.workspace_bytes(Q, m),), 0xFF, dtype=torch.uint8, device="cuda")
        assert torch.equal(f8.gemm(Q, x, out_dtype=dt, workspace=ws), want)
        wide = torch.zeros(m, k + 3, dtype=DT[dtype], device="cuda")
        wide[:, :k] = x
        assert torch.equal(f8.gemm(Q, wide[:, :k], out_dtype=dt), want)


def test_more_tokens_than_a_grid_dimension():
    # 65536 workgroups of 64 tokens and one more panel: the tokens of a narrow
    # weight do not fit the second dimension of a grid
    m, n, k = 65536 * 64 + 16, 16, 16
    W, X = f8.pack(normal(60, n, k, "bf16")), f8.quant(normal(61, m, k, "bf16"))
    for out in (torch.float32, torch.bfloat16):
        y = f8.gemm(W, X, out_dtype=out)
        x8, w8 = as64(f8.unpack(X, out_dtype=torch.float32)), as64(f8.unpack(W, out_dtype=torch.float32))
        ref, size = x8 @ w8.T, np.abs(x8) @ np.abs(w8.T)
        bound = k * 2.0 ** -23 * size + HALF[out] * np.abs(ref)
        if out != torch.float32:
            bound += 2.0 ** -11 * np.abs(x8).max(1, keepdims=True) * np.abs(w8).max(1)[None]
        assert (np.abs(as64(y) - ref) <= bound).all()
