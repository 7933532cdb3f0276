"""The 4-bit read-back of weights on either side of 256 MiB, where its 16-bit outputs
begin to go around the caches, takes about as long a byte (fp32 ones that did so took
twice as long).  Least times of interleaved calls; half as much again is allowed."""
import pytest
import torch

from matmul_pack_b1_amd import q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_time_a_byte(dtype):
    k = 8192
    rows = [(250 << 20) // (k * dtype.itemsize), (262 << 20) // (k * dtype.itemsize)]
    Qs = [q4.pack(torch.randn(n, k, device="cuda", dtype=torch.bfloat16)) for n in rows]
    outs = [torch.empty(n, k, dtype=dtype, device="cuda") for n in rows]
    least = [float("inf")] * 2
    for turn in range(25):
        for i in range(2):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(4):
                q4.unpack(Qs[i], out=outs[i])
            end.record()
            end.synchronize()
            if turn >= 5:
                least[i] = min(least[i], start.elapsed_time(end) / rows[i])
    assert least[1] < 1.5 * least[0], least
