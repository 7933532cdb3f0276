"""The norm over a list of tensors, and clipping by it, on the GPU against
float64.

Squares are summed in 64 bits (an error of at most count * 2^-53, relative), so
the norm is off by its rounding to fp32: 2^-24, relative.  The factor is
max_norm / (norm + 1e-6) in 64 bits, rounded to fp32 (2^-24), the product is
rounded to fp32 (2^-24) and to the tensor's type."""
import math

import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import clip

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def normal(seed, shape, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).cuda()


def as64(t):
    return t.detach().cpu().double().numpy()


def reference(tensors, max_norm):
    norm = math.sqrt(sum(float(np.square(as64(t)).sum()) for t in tensors))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def check(tensors, max_norm, got, norm):
    ref, factor = reference(tensors, max_norm)
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    for a, b in zip(tensors, got):
        want = as64(a) * factor
        tol = (2.0 ** -22 + HALF[b.dtype]) * np.abs(want) + LEAST[b.dtype]
        assert (np.abs(as64(b) - want) <= tol).all()
        if factor == 1.0:
            assert torch.equal(a, b)


SIZES = [(1,), (7,), (8,), (255, 3), (1024,), (16384,), (16385,), (333, 257), (5, 40000)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SIZES)
@pytest.mark.parametrize("max_norm", [0.5, 1e6, 0.0])
def test_one_tensor(dtype, shape, max_norm):
    t = normal(1, shape, dtype)
    before = t.clone()
    assert abs(float(clip.norm([t])) - reference([t], 1)[0]) <= 2.0 ** -23 * reference([t], 1)[0]
    out = torch.full_like(t, 7.0)
    norm = clip.clip([t], max_norm, outs=[out])
    assert torch.equal(t, before)
    check([before], max_norm, [out], norm)
    again = clip.clip([t], max_norm)
    assert torch.equal(again, norm) and torch.equal(t, out)


@pytest.mark.parametrize("count", [2, 63, 64, 65, 200])
@pytest.mark.parametrize("max_norm", [1.0, 1e9])
def test_many_tensors(count, max_norm):
    rng = np.random.default_rng(count)
    ts = [normal(i, (int(rng.integers(1, 3000)),), ("bf16", "f16", "f32")[i % 3]) for i in range(count)]
    before = [t.clone() for t in ts]
    norm = clip.clip(ts, max_norm)
    check(before, max_norm, ts, norm)
    assert float(clip.norm(before)) == float(norm)


def test_large_tensors():
    ts = [normal(1, (4096, 4097), "bf16", 1e-3), normal(2, (3000001,), "f32", 1e-3)]
    before = [t.clone() for t in ts]
    check(before, 1.0, ts, clip.clip(ts, 1.0))


@pytest.mark.parametrize("scale", [1e-30, 1e25, 3e37])
def test_sums_neither_overflow_nor_vanish(scale):
    ts = [normal(3, (5000,), "f32", scale), normal(4, (3001,), "bf16", scale)]
    ref, _ = reference(ts, 1.0)
    got = float(clip.norm(ts))
    if ref > 3.4028235677973366e38:      # halfway past the largest fp32
        assert math.isinf(got)
    else:
        assert abs(got - ref) <= 2.0 ** -23 * ref
    outs = [torch.empty_like(t) for t in ts]
    check(ts, 1.0, outs, clip.clip(ts, 1.0, outs=outs)) if ref < 3e38 else None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_apart(dtype):
    """Strided rows on either side; what lies between them stays."""
    base = torch.full((40, 301), 9.0, dtype=DT[dtype], device="cuda")
    t = base[1:38, 3:270]
    t.copy_(normal(5, (37, 267), dtype))
    flat = t.contiguous()
    want = torch.empty_like(flat)
    norm = clip.clip([flat], 1.0, outs=[want])
    assert abs(float(clip.norm([t])) - float(norm)) <= 2.0 ** -23 * float(norm)
    out = torch.full((40, 275), 9.0, dtype=DT[dtype], device="cuda")
    for data, to in ((t, out[2:39, 1:268]), (flat, out[2:39, 1:268]), (t, torch.empty_like(flat))):
        clip.clip([data], 1.0, outs=[to])
        assert torch.equal(to, want)
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[2:39, 1:268] = False
    assert bool((out[rest] == 9.0).all())
    clip.clip([t], 1.0)
    assert torch.equal(t, want)
    rest = torch.ones_like(base, dtype=torch.bool)
    rest[1:38, 3:270] = False
    assert bool((base[rest] == 9.0).all())


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_unaligned(offset, dtype):
    base = normal(6, (20000,), dtype)
    t = base[offset:19990]
    before = base.clone()
    out = torch.full((20010,), 9.0, dtype=DT[dtype], device="cuda")
    check([t], 1.0, [out[7:7 + t.numel()]], clip.clip([t], 1.0, outs=[out[7:7 + t.numel()]]))
    clip.clip([t], 1.0)
    assert torch.equal(t, out[7:7 + t.numel()])
    assert torch.equal(base[:offset], before[:offset]) and torch.equal(base[19990:], before[19990:])
    assert bool((out[:7] == 9.0).all()) and bool((out[7 + t.numel():] == 9.0).all())


def test_not_finite():
    t = normal(7, (3000,), "f32")
    t[17] = float("nan")
    u = normal(8, (100,), "bf16")
    assert math.isnan(float(clip.norm([u, t])))
    outs = [torch.zeros_like(u), torch.zeros_like(t)]
    assert math.isnan(float(clip.clip([u, t], 1.0, outs=outs)))
    assert all(bool(o.isnan().all()) for o in outs)
    t[17] = float("inf")
    assert math.isinf(float(clip.clip([u, t], 1.0, outs=outs)))
    assert bool((outs[0] == 0).all()) and bool(outs[1][17].isnan()) and int(outs[1].isnan().sum()) == 1


def test_empty():
    assert float(clip.norm([])) == 0.0
    assert float(clip.clip([], 1.0)) == 0.0
    e = torch.empty(0, 5, device="cuda")
    assert float(clip.clip([e, e], 1.0)) == 0.0
    t = normal(1, (100,), "f32")
    assert float(clip.norm([e, t, e])) == float(clip.norm([t]))


def test_same_tensor_twice_counts_twice_in_the_norm():
    t = normal(1, (1000,), "f32")
    assert abs(float(clip.norm([t, t])) - math.sqrt(2) * reference([t], 1)[0]) < 1e-5
    with pytest.raises(RuntimeError, match="overlaps"):
        clip.clip([t, t], 1.0)


def test_graph_capture():
    ts = [normal(i, (3000 + 17 * i,), ("bf16", "f32")[i % 2]) for i in range(70)]
    outs = [torch.empty_like(t) for t in ts]
    norm = torch.empty((), device="cuda")
    clip.clip(ts, 1.0, outs=outs, out=norm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clip.clip(ts, 1.0, outs=outs, out=norm)
    for seed in range(3):
        for i, t in enumerate(ts):
            t.copy_(normal(100 * seed + i, t.shape, "f32", 10.0 ** (-2 * seed)))
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(t) for t in ts]
        assert torch.equal(clip.clip(ts, 1.0, outs=want), norm)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        check(ts, 1.0, outs, norm)


def test_another_stream_and_own_workspace():
    ts = [normal(i, (50000,), "bf16") for i in range(3)]
    want = clip.norm(ts)
    ws = torch.full((clip.workspace_bytes(ts),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = clip.norm(ts, workspace=ws)
    side.synchronize()
    assert torch.equal(want, got)
    with pytest.raises(RuntimeError, match="workspace"):
        clip.norm(ts, workspace=ws[:8])
