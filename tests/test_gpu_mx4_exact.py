"""The MX4 linear layer on whole numbers, where nothing may round: elements of X
and W are -1, 0 or 1, T, G and the adapter's entries small whole numbers, so
every value is exact in its type and every sum of products, in any order and
any split, a whole number below 2^24.  Y, T and the gradients are then one
rounding of the exact result to bf16, and are compared bit for bit.

T B^T and G A are as large as the frozen product: results without them differ
almost everywhere, which each test checks on the reference."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from tests.gpu_util import DEV, guarded_like

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _signs(g, *shape):
    return g.integers(-1, 2, shape).astype(np.float64)


def _sparse(g, rows, cols, each):
    """Rows of signs with at most `each` entries that are not 0."""
    a = np.zeros((rows, cols))
    for r in range(rows):
        at = g.permutation(cols)[:each]
        a[r, at] = g.choice((-1.0, 1.0), at.size)
    return a


def _small(g, *shape):
    return g.integers(1, 9, shape) * g.choice((-1.0, 1.0), shape)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(BF16).to(DEV)


def _rounded(a):
    """bf16 of whole numbers: fp32 holds them, then one rounding to nearest even."""
    assert np.abs(a).max() < 2 ** 24 and (a == np.round(a)).all()
    return torch.from_numpy(a.astype(np.float32)).to(BF16)


def _equal(got, want, name):
    want = _rounded(want)
    bad = torch.nonzero(got.cpu().float() != want.float())
    assert bad.numel() == 0, (name, bad.shape[0], bad[:5].tolist(), got.cpu()[tuple(bad[0])], want[tuple(bad[0])])


def _matters(whole, without):
    assert (_rounded(whole) != _rounded(without)).float().mean() > 0.5, "the adapter's part is lost in the rounding"


FORWARD = [(1, 4096, 4096, 64), (4, 200, 288, 16), (17, 136, 512, 128), (64, 1024, 11008, 64), (65, 1, 16384, 1),
           (70, 1001, 11008, 8), (75, 552, 8224, 64), (128, 136, 22016, 64), (200, 264, 5632, 100), (300, 330, 8192, 33),
           (2047, 72, 1056, 64), (2050, 64, 1056, 5), (2081, 128, 320, 33), (2049, 8200, 288, 64), (2100, 24, 96, 128)]


@pytest.mark.parametrize("M,N,K,r", FORWARD)
def test_forward(M, N, K, r):
    g = np.random.default_rng(M + N + K + r)
    X, W = _signs(g, M, K), _signs(g, N, K)
    A, B = _sparse(g, r, K, 60), _small(g, N, r)
    T, frozen = X @ A.T, X @ W.T
    want = frozen + T @ B.T
    _matters(want, frozen)
    w = q.MX4Tensor.quantize(_dev(W))
    gy, Y = guarded_like((M, N), BF16, 1)
    gt, Tg = guarded_like((M, r), BF16, 2)
    q.mx4_linear_fwd(_dev(X), w, _dev(A), _dev(B), 1.0, T_out=Tg, out=Y)
    _equal(Tg, T, "T")
    _equal(Y, want, "Y")
    assert gy.intact() and gt.intact()
    Y2, _ = q.mx4_linear_fwd(_dev(X), w, _dev(A), _dev(B), 2.0)
    _equal(Y2, want + T @ B.T, "Y at twice the scale")
    _equal(q.mx4_matmul(q.MX4Tensor.quantize(_dev(X)), w, _dev(T), _dev(B)), want, "product")


BACKWARD = [(1, 4096, 64, 8), (69, 2240, 2560, 64), (75, 576, 1344, 33), (200, 1024, 192, 100), (513, 1344, 704, 64),
            (33, 22016, 128, 1), (128, 512, 320, 128), (128, 11008, 4096, 64), (1100, 256, 4096, 64), (700, 320, 2048, 16),
            (300, 192, 4096, 64), (4096, 1024, 4096, 64), (4099, 256, 4160, 8)]


@pytest.mark.parametrize("M,N,K,r", BACKWARD)
def test_backward(M, N, K, r):
    g = np.random.default_rng(M + N + K + r)
    dY, X, W = _signs(g, M, N), _signs(g, M, K), _signs(g, N, K)
    A, B, T = _small(g, r, K), _sparse(g, r, N, 60).T, _small(g, M, r)
    G, frozen = dY @ B, dY @ W
    _matters(frozen + G @ A, frozen)
    w = q.MX4Tensor.quantize(_dev(W))
    guards = [guarded_like(s, BF16, i) for i, s in enumerate(((M, K), (r, K), (N, r)))]
    dX, dA, dB = (t for _, t in guards)
    q.mx4_linear_bwd(_dev(dY), _dev(X), _dev(T), w, _dev(A), _dev(B), 1.0, dX_out=dX, dA_out=dA, dB_out=dB)
    _equal(dX, frozen + G @ A, "dX")
    _equal(dA, G.T @ X, "dA")
    _equal(dB, dY.T @ T, "dB")
    assert all(gd.intact() for gd, _ in guards)
