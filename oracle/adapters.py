"""The linear layer with many adapters, and the gradient norm, in float64 by their
definitions (test infrastructure only)."""

import numpy as np


def forward(X, W, A, B, scale, index):
    """(Y [M, N], T [M, r]) of X [M, K], W [N, K], A [n, r, K], B [n, N, r]."""
    Y, T = X @ W.T, np.zeros((X.shape[0], A.shape[1]))
    for m, a in enumerate(index):
        if 0 <= a < A.shape[0]:
            T[m] = scale[a] * (A[a] @ X[m])
            Y[m] += B[a] @ T[m]
    return Y, T


def backward(dY, X, W, A, B, scale, index):
    """(dX, dA, dB) for the gradient dY [M, N]."""
    dX, dA, dB = dY @ W, np.zeros(A.shape), np.zeros(B.shape)
    for m, a in enumerate(index):
        if 0 <= a < A.shape[0]:
            G = scale[a] * (dY[m] @ B[a])
            dX[m] += G @ A[a]
            dA[a] += np.outer(G, X[m])
            dB[a] += np.outer(dY[m], scale[a] * (A[a] @ X[m]))
    return dX, dA, dB


def clip(grads, max_norm, groups=1):
    """(norms [groups], clipped gradients): every tensor is cut along its first axis into `groups` equal parts."""
    norm = np.zeros(groups)
    for g in grads:
        norm += (np.asarray(g, np.float64).reshape(groups, -1) ** 2).sum(1)
    norm = np.sqrt(norm)
    with np.errstate(invalid="ignore"):
        coef = np.where(np.isnan(norm), np.nan, np.minimum(1.0, max_norm / (norm + 1e-6)))
    return norm, [(np.asarray(g, np.float64).reshape(groups, -1) * coef[:, None]).reshape(np.shape(g)) for g in grads]
