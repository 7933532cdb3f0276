"""CPU reference of the gated projection and its gradients (NumPy, float64);
test infrastructure only, shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[float])


def act(g, kind):
    """(activation, derivative) of each element."""
    g = np.asarray(g, np.float64)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s + g * s * (1.0 - s)
    if kind == "gelu":
        phi = 0.5 * _erfc(-g / math.sqrt(2.0))
        return g * phi, phi + g * np.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def forward(x, wg, wu, kind):
    """G, U, H."""
    x, wg, wu = (np.asarray(a, np.float64) for a in (x, wg, wu))
    g, u = x @ wg.T, x @ wu.T
    return g, u, act(g, kind)[0] * u


def gradients(g, u, dh, kind):
    """dG, dU."""
    a, slope = act(g, kind)
    return dh * u * slope, dh * a
