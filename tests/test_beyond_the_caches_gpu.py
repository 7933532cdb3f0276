"""What is read or written in more than the last-level cache's 256 MiB takes loads
and stores of its own: clipping, and the 4-bit read-back."""
import math

import pytest
import torch

from matmul_pack_b1_amd import clip, q4

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def fill(t, seed):
    return t.copy_(torch.randn(t.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * 1e-3)


def pieces(few):
    """Tensors of over 256 MiB in all: three types, element-aligned, ragged, rows
    apart; more than `few` go into the larger table of a launch."""
    guard = 13
    base16 = torch.full((60_000_011 + 2 * guard,), 9.0, dtype=torch.bfloat16, device="cuda")
    half = torch.full((20_000_003 + 2 * guard,), 9.0, dtype=torch.float16, device="cuda")
    base32 = torch.full((1025, 40_011), 9.0, dtype=torch.float32, device="cuda")
    out = [base16[guard:-guard], half[guard:-guard], base32[1:, 3:40_004], torch.empty(16_385, device="cuda")]
    if not few:
        out += [torch.empty(1000 + i, dtype=torch.bfloat16, device="cuda") for i in range(70)]
    assert sum(t.numel() * t.element_size() for t in out) > 256 << 20
    return (base16, half, base32), [fill(t, i) for i, t in enumerate(out)]


def untouched(bases):
    base16, half, base32 = bases
    rest = torch.ones_like(base32, dtype=torch.bool)
    rest[1:, 3:40_004] = False
    return (all(bool((b[:13] == 9.0).all()) and bool((b[-13:] == 9.0).all()) for b in (base16, half))
            and bool((base32[rest] == 9.0).all()))


@pytest.mark.parametrize("few", [True, False])
def test_clip(few):
    bases, ts = pieces(few)
    before = [t.clone() for t in ts]
    ref = math.sqrt(sum(float(t.double().square().sum()) for t in ts))
    factor = 0.25 / (ref + 1e-6)
    assert factor < 1
    assert abs(float(clip.norm(ts)) - ref) <= 2.0 ** -23 * ref
    others, outs = pieces(few)
    norm = clip.clip(ts, 0.25, outs=outs)
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    for t, b, o in zip(ts, before, outs):
        assert torch.equal(t, b)
        want = b.double() * factor
        assert bool(((o.double() - want).abs() <= (2.0 ** -22 + HALF[o.dtype]) * want.abs() + LEAST[o.dtype]).all())
    assert untouched(others)
    assert torch.equal(clip.clip(ts, 0.25), norm)          # in place: the same
    assert all(torch.equal(t, o) for t, o in zip(ts, outs))
    assert untouched(bases)
    again = [t.clone() for t in ts]
    clip.clip(ts, 1e9)                                     # a factor of 1
    assert all(torch.equal(t, a) for t, a in zip(ts, again))
    clip.clip(ts, 1e9, outs=outs)
    assert all(torch.equal(o, a) for o, a in zip(outs, again))


# columns, row stride and first element: rows that begin anywhere, or at 64 bytes
@pytest.mark.parametrize("k,pitch,offset", [(8195, 8197, 1), (8195, 8224, 32), (8192, 8192, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_q4_read_back(dtype, k, pitch, offset):
    """The same values as from slices of the rows, which are read back through the
    caches."""
    n = (256 << 20) // (k * dtype.itemsize) + 3
    w = torch.randn(n, k, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    base = torch.full((n * pitch + offset + 99,), 7.0, dtype=dtype, device="cuda")
    assert base.data_ptr() % 64 == 0
    out = torch.as_strided(base, (n, k), (pitch, 1), offset)
    q4.unpack(q4.pack(w), out=out)
    for r in range(0, n, 5000):
        part = q4.unpack(q4.pack(w[r:r + 5000]), out_dtype=dtype)
        assert part.numel() * part.element_size() <= 256 << 20
        assert torch.equal(out[r:r + 5000], part)
    out.fill_(7.0)
    assert bool((base == 7.0).all())
