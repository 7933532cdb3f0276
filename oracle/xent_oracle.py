"""CPU reference of the softmax cross entropy over a vocabulary projection
(NumPy, float64); test infrastructure only, shares no code with the library."""
from __future__ import annotations

import numpy as np


def cross_entropy(x, w, target, n_vocab, grad=None, ignore=-100):
    """loss, lse (0 where the target is `ignore`) and, with grad, dx and dw:
    z = x w^T over the first n_vocab rows of w, loss = log sum exp z -
    z[target], dz = grad (softmax z - onehot)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    seen = target != ignore
    xs = np.where(seen[:, None], x, 0.0)
    z = xs @ w[:n_vocab].T
    top = z.max(axis=1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    rows = np.arange(len(target))[seen]
    loss = np.zeros(len(target))
    loss[rows] = lse[rows] - z[rows, target[rows]]
    if grad is None:
        return loss, np.where(seen, lse, 0.0)
    g = np.exp(z - lse[:, None])
    g[rows, target[rows]] -= 1.0
    g[~seen] = 0.0
    dz = g * np.where(seen, grad, 0.0)[:, None]
    dw = np.zeros_like(w)
    dw[:n_vocab] = dz.T @ xs
    return loss, np.where(seen, lse, 0.0), dz @ w[:n_vocab], dw
