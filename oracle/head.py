"""Softmax cross entropy through an output head in float64, by its definition
(test infrastructure only)."""

import numpy as np

from . import vocab


def cross_entropy(X, W, target, weight):
    """(loss [M], log-sum-exp [M], p [M, V], dX, dW) of X [M, K], W [V, K]; rows
    whose target is outside [0, V) take no part, whatever they hold."""
    M, V = X.shape[0], W.shape[0]
    real = (target >= 0) & (target < V)
    z = np.where(real[:, None], X, 0.0) @ W.T
    lp = vocab.log_softmax(z)
    at = np.where(real, target, 0)
    rows = np.arange(M)
    loss = np.where(real, -lp[rows, at], 0.0)
    lse = np.where(real, z[rows, at] - lp[rows, at], 0.0)
    p = np.exp(lp)
    d = p.copy()
    d[rows, at] = np.expm1(lp[rows, at])
    d *= np.where(real, weight, 0.0)[:, None]
    return loss, lse, p, d @ W, d.T @ np.where(real[:, None], X, 0.0)
