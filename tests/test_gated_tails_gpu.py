"""The tails of the gated projection's activations and of their slopes.

G is one product of the call here, so its value is exact, and every other product
is by a power of two: what is off is act (or its slope) and the roundings to 16 bits.
fp32 errors relative to a value, for the formulas of the header with one rounding an
operation and 2^-23 for an exponential or a reciprocal:
  silu       (|g| + 4) * 2^-22: the exponential's argument is off by |g| 2^-23
  gelu_tanh  (4 y + 8) * 2^-23, y = 2 c |g| (1 + 0.0447 g^2) the argument, in four
             roundings and one for its multiple by log2 e
  gelu       (2.5 g^2 + 12) * 2^-23: x^2 = g^2 / 2 with x off by 2^-23, the sum in the
             exponent rounded at x^2, and 1.2e-7 of the fit
A slope is a sum of two terms, each off by that much of itself."""
import math

import numpy as np
import pytest
import torch

from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated, q4
from oracle import gated_oracle as go

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DENSE = np.zeros((2, 1), dtype=np.uint8)

# 128 gates of eight bits: tails down to where act leaves fp32's normal numbers, and
# the middle
TAIL = {"silu": 80.0, "gelu": 12.5, "gelu_tanh": 8.5}


def exact(g, act):
    """(act, slope) in float64.  (1 + tanh, as the oracle has it, loses the tail.)"""
    if act != "gelu_tanh":
        return go.act(g, act)
    c = math.sqrt(2.0 / math.pi)
    s = 1.0 / (1.0 + np.exp(-2.0 * c * (g + 0.044715 * g ** 3)))
    return g * s, s + g * s * (1.0 - s) * 2.0 * c * (1.0 + 3.0 * 0.044715 * g * g)


def gates(act, positive):
    g = -np.geomspace(2.0 ** -9, TAIL[act], 128)
    if positive:
        g[::2] *= -1
    return torch.from_numpy(g).to(torch.bfloat16).double()


def act_eps(g, act):
    g = np.abs(g)
    if act == "silu":
        return (g + 4.0) * 2.0 ** -22
    if act == "gelu_tanh":
        return (4.0 * 2.0 * math.sqrt(2.0 / math.pi) * g * (1.0 + 0.044715 * g * g) + 8.0) * 2.0 ** -23
    return (2.5 * g * g + 12.0) * 2.0 ** -23


def one_column(values, column, kind, dtype):
    """A weight of 128 x 64 with `values` in a column: packed dense or in 4 bits."""
    w = torch.zeros(128, 64, dtype=torch.float64)
    w[:, column] = values
    w = w.to(dtype).cuda()
    assert torch.equal(w[:, column].double().cpu(), values)
    return hb.pack(w, DENSE, 64, 64, "idx2") if kind == "packed" else q4.pack(w)


@pytest.mark.parametrize("m", [1, 5, 40, 140])
@pytest.mark.parametrize("act", list(gated.ACTS))
@pytest.mark.parametrize("kind", ["packed", "4bit"])
def test_tails(act, kind, m):
    """Gates from x, eight bits each, in bf16 (whose range holds every H)."""
    vals = gates(act, True)
    if kind == "4bit":   # one code a gate: 6 2^e and 4 2^e, e down to where the tail ends
        e = torch.arange(128) // 2 % 9 - 6
        vals = torch.where(torch.arange(128) % 2 == 0, 6.0, 4.0) * 2.0 ** e.double()
        vals = torch.where(vals <= TAIL[act], vals, vals / 16)
        vals[torch.arange(128) % 3 > 0] *= -1
    G = one_column(vals, 3, kind, torch.bfloat16)
    U = one_column(torch.full((128,), 2.0, dtype=torch.float64), 9, kind, torch.bfloat16)
    x = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 3], x[:, 9] = 1.0, 0.5
    h = gated.forward(G, U, x, act=act).double().cpu().numpy()
    g = vals.numpy()
    ref = exact(g, act)[0]
    tol = np.abs(ref) * (2.0 ** -8 + 2 * act_eps(g, act)) + 2.0 ** -126
    assert (np.abs(h - ref) <= tol).all(), (g[(np.abs(h - ref) > tol).any(0)][:8], act)


@pytest.mark.parametrize("m", [1, 5, 40, 140])
@pytest.mark.parametrize("act", list(gated.ACTS))
def test_tails_in_fp16(act, m):
    """Eleven bits: u = 2^30 brings the tail down to 2^-44 into fp16."""
    vals = gates(act, False)
    ref = exact(vals.numpy(), act)[0]
    lift = np.clip(-np.floor(np.log2(np.abs(ref))), 1, 30)
    G = one_column(vals, 3, "packed", torch.float16)
    U = one_column(torch.from_numpy(2.0 ** (lift - 15)), 9, "packed", torch.float16)
    x = torch.zeros(m, 64, dtype=torch.float16, device="cuda")
    x[:, 3], x[:, 9] = 1.0, 2.0 ** 15
    h = gated.forward(G, U, x, act=act).double().cpu().numpy()
    ref = ref * 2.0 ** lift
    tol = np.abs(ref) * (2.0 ** -11 + 2 * act_eps(vals.numpy(), act)) + 2.0 ** -25
    assert (np.abs(h - ref) <= tol).all(), (vals.numpy()[(np.abs(h - ref) > tol).any(0)][:8], act)


@pytest.mark.parametrize("m", [1, 70, 300])
@pytest.mark.parametrize("act", list(gated.ACTS))
def test_slopes_tails(act, m):
    """dG and dU of one token, through dW of its one activation."""
    vals = gates(act, True)
    g = vals.float().repeat(m, 1).cuda()
    u = torch.full((m, 128), 2.0, device="cuda")
    dh = torch.zeros(m, 128, dtype=torch.bfloat16, device="cuda")
    dh[m - 1] = 0.5
    x = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda")
    x[m - 1, 7] = 1.0
    P = one_column(vals, 3, "packed", torch.bfloat16)
    dx, dwg, dwu = gated.backward(P, P, x, g, u, dh, act=act, need_dw=True)
    gn = vals.numpy()
    a, slope = exact(gn, act)
    # the slope's two terms: act / g, and the rest
    terms = np.abs(a / gn) + np.abs(slope - a / gn)
    eps = 2 * act_eps(gn, act)
    for got, ref, err in ((dwg, slope, eps * terms), (dwu, 0.5 * a, eps * np.abs(0.5 * a))):
        got = got.double().cpu().numpy()
        # rounded to bf16 as a gradient; once more, to itself, as the output
        assert (np.abs(got[:, 7] - ref) <= np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -7) + err * 1.01 + 2.0 ** -126).all()
        assert not got[:, :7].any() and not got[:, 8:].any()
