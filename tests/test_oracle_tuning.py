"""Pins of the oracle's adapter layer, head loss and gradient norm against closed
forms, differences and an independent routine."""

import numpy as np
import torch

from oracle import adapters, head


def test_adapters_against_a_block_matrix_and_differences():
    g = np.random.default_rng(0)
    M, N, K, n, r = 9, 5, 7, 3, 2
    X, W, A, B, s = (g.standard_normal(v) for v in ((M, K), (N, K), (n, r, K), (n, N, r), (n,)))
    idx = np.array([0, 2, -1, 1, 1, 3, 0, 2, 2])
    Y, T = adapters.forward(X, W, A, B, s, idx)
    eff = [W + (s[a] * B[a] @ A[a] if 0 <= a < n else 0) for a in idx]
    np.testing.assert_allclose(Y, np.stack([e @ x for e, x in zip(eff, X)]), rtol=1e-12)
    assert not T[2].any() and not T[5].any()
    dY = g.standard_normal((M, N))
    grads = adapters.backward(dY, X, W, A, B, s, idx)
    for k, (v, grad) in enumerate(zip((X, A, B), grads)):
        d = g.standard_normal(v.shape)
        f = []
        for h in (1e-6, -1e-6):
            args = [X, A, B]
            args[k] = v + h * d
            f.append((adapters.forward(args[0], W, args[1], args[2], s, idx)[0] * dY).sum())
        np.testing.assert_allclose((grad * d).sum(), (f[0] - f[1]) / 2e-6, rtol=1e-6)


def test_head_against_torch():
    g = np.random.default_rng(1)
    X, W = g.standard_normal((6, 8)), g.standard_normal((11, 8))
    t = np.array([3, -100, 10, 0, 11, 5])
    weight = g.standard_normal(6)
    loss, lse, p, dX, dW = head.cross_entropy(X, W, t, weight)
    x, w = torch.tensor(X, requires_grad=True), torch.tensor(W, requires_grad=True)
    tt = torch.tensor(np.where(t == 11, -100, t))
    want = torch.nn.functional.cross_entropy(x @ w.t(), tt, reduction="none")
    (want * torch.tensor(weight)).sum().backward()
    np.testing.assert_allclose(loss, want.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(dX, x.grad.numpy(), rtol=1e-10, atol=1e-14)
    np.testing.assert_allclose(dW, w.grad.numpy(), rtol=1e-10, atol=1e-14)
    real = (t >= 0) & (t < 11)
    np.testing.assert_allclose(lse[real], torch.logsumexp(x @ w.t(), 1).detach().numpy()[real], rtol=1e-12)
    X[1] = np.nan                                     # no target: whatever it holds
    again = head.cross_entropy(X, W, t, weight)
    for k in (0, 1, 3, 4):
        np.testing.assert_array_equal(again[k], (loss, lse, p, dX, dW)[k])


def test_clip_against_torch():
    g = torch.Generator().manual_seed(2)
    ps = [torch.nn.Parameter(torch.zeros(s, dtype=torch.float64)) for s in ((4, 3), (5,), (2, 2, 2))]
    for p in ps:
        p.grad = torch.randn(p.shape, generator=g, dtype=torch.float64)
    norm, want = adapters.clip([p.grad.numpy() for p in ps], 0.7)
    got = torch.nn.utils.clip_grad_norm_(ps, 0.7)
    np.testing.assert_allclose(norm, [got.item()], rtol=1e-12)
    for p, w in zip(ps, want):
        np.testing.assert_allclose(p.grad.numpy(), w, rtol=1e-12)
    norm, out = adapters.clip([np.array([[3.0], [0.1]]), np.array([4.0, 0.0])], 1.0, groups=2)
    np.testing.assert_allclose(norm, [5.0, 0.1])
    np.testing.assert_allclose(out[0], [[0.6], [0.1]], rtol=1e-6)
