"""The larger kernels of the 4-bit products and of the gated projection captured into
graphs before any eager call of theirs here, and replayed on new inputs with eager
calls between; and on two streams at once."""
import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated, q4

pytestmark = pytest.mark.gpu


def normal(seed, rows, cols, dtype, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(dtype)


def packed(seed, n, k, dtype):
    tiles = (np.arange(n // 64 * (k // 64)) % 2).astype(np.uint8)
    return hb.pack(normal(seed, n, k, dtype, k ** -0.5), tiles, 64, 64, "idx2")


def replayed(inputs, call):
    """call() captured; three replays, each on other inputs, against call() eager."""
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for seed in range(3):
        for i, t in enumerate(inputs):
            t.copy_(normal(10 * seed + i, *t.shape, t.dtype, 0.1 ** seed))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, call()):
            assert torch.equal(a, b)


# k shared by token blocks, in parts; tiles whole and cut (route_shapes.py)
@pytest.mark.parametrize("n,k,m", [(1100, 2100, 301), (8200, 515, 901), (4097, 515, 1003), (8200, 3100, 401)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_products(n, k, m, dtype):
    Q, x = q4.pack(normal(1, n, k, dtype, 0.05)), normal(2, m, k, dtype)
    replayed([x], lambda: [q4.gemm(Q, x)])


@pytest.mark.parametrize("n,k,m", [(64, 768, 129), (2816, 1024, 333), (3200, 2560, 401), (2816, 4096, 261)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradients(n, k, m, dtype):
    G, U = packed(1, n, k, dtype), packed(2, n, k, dtype)
    x, dh = normal(3, m, k, dtype), normal(4, m, n, dtype, 0.1)

    def call():
        h, g, u = gated.forward(G, U, x, save=True)
        return (h, g, u) + gated.backward(G, U, x, g, u, dh, need_dw=True)
    replayed([x, dh], call)


def test_two_streams():
    """A training step and a 4-bit product, several of each under way."""
    n, k, m = 2816, 1024, 333
    G, U = packed(1, n, k, torch.bfloat16), packed(2, n, k, torch.bfloat16)
    x, dh = normal(3, m, k, torch.bfloat16), normal(4, m, n, torch.bfloat16, 0.1)
    Q, z = q4.pack(normal(5, 8200, 515, torch.bfloat16, 0.05)), normal(6, 901, 515, torch.bfloat16)

    def step():
        h, g, u = gated.forward(G, U, x, save=True)
        return (h,) + gated.backward(G, U, x, g, u, dh, need_dw=True)
    want, want4 = step(), q4.gemm(Q, z)
    torch.cuda.synchronize()
    streams, got, got4 = [torch.cuda.Stream() for _ in range(2)], [], []
    for _ in range(4):
        with torch.cuda.stream(streams[0]):
            got.append(step())
        with torch.cuda.stream(streams[1]):
            got4.append(q4.gemm(Q, z))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    assert all(torch.equal(y, want4) for y in got4)
