"""Infinite norms and an infinite max_norm (hyb_clip.h)."""
import math

import pytest
import torch

from matmul_pack_b1_amd import clip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinities(dtype):
    t = torch.randn(5000, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    before, out = t.clone(), torch.empty_like(t)
    norm = clip.clip([t], math.inf, outs=[out])             # nothing is clipped
    assert math.isfinite(float(norm)) and torch.equal(out, t)
    clip.clip([t], math.inf)
    assert torch.equal(t, before)
    t[7] = -math.inf
    assert float(clip.clip([t], 3e38, outs=[out])) == math.inf
    assert bool(out[7].isnan()) and int((out == 0).sum()) == 4999
    assert float(clip.clip([t], math.inf, outs=[out])) == math.inf
    assert bool(out.isnan().all())
