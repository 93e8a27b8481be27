"""The head's gradient from up to 64 rows on the GPU against float64: within its own rounding to bf16.

Logits are whole numbers, exact in fp32.  A dz_mj is off by the 2^-19 + 2^-22 of its p_mj (exponential and
reference), and by 2^-16 of itself where two bf16 numbers hold it (each rounding 2^-8); the fp32
sum of 2 M terms adds 2 M 2^-23 of them, the result's rounding 2^-8, and what is below 2^-126 may be 0."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from oracle import head as ohead
from tests import test_gpu_head as head

pytestmark = pytest.mark.gpu

R, S = 2.0 ** -8, 2.0 ** -23


@pytest.mark.parametrize("M,V,K", [(1, 1, 64), (1, 300, 64), (1, 5003, 1088), (2, 129, 192), (7, 1000, 128), (40, 4136, 4096), (63, 65, 320),
                                   (64, 2049, 128)])
def test_the_gradient_is_off_by_its_own_rounding(M, V, K):
    for seed in range(3):
        X, W, t, weight = head._case(M, V, K, seed=seed, whole=True)
        x, g = head._f64(X), head._f64(weight)
        tt = t.cpu().numpy()
        _, _, p, _, want = ohead.cross_entropy(x, head._f64(W), tt, g)
        real = (tt >= 0) & (tt < V)
        at = np.where(real, tt, 0)
        d = p.copy()
        d[np.arange(M), at] = 1 - p[np.arange(M), at]
        ag = np.where(real, np.abs(g), 0)[:, None]
        xa = np.abs(x)
        e = ((2.0 ** -16 + 2 * M * S) * d * ag + (2.0 ** -19 + 2.0 ** -22) * p * ag).T @ xa + 2.0 ** -126 * (2 + 2 * xa.sum(0))
        lse = q.head_cross_entropy_fwd(X, W, t)[1]
        dW = q.head_cross_entropy_dW(X, W, t, lse, weight)
        head._close(dW, want, R * (np.abs(want) + e) + e, "dW")
        assert torch.equal(dW, q.head_cross_entropy_dW(X, W, t, lse, weight))


@pytest.mark.parametrize("M", [3, 64])
def test_infinite_weights_stay_infinite(M):
    """A row's weight of infinity, and of a size whose rounding to bf16 overflows, is infinite and no NaN where its row is not 0."""
    X, W, t, weight = head._case(M, 2000, 64, seed=1, whole=True, ignored=0)
    X[:] = 1.0
    W[:, 1:] = 0
    W[:, 0] = 0                                            # p = 1/2000: dz_t = -1999/2000 weight
    weight[:] = 0
    weight[1] = torch.finfo(torch.float32).max          # dz_t is past 3.396e38, where bf16 ends
    weight[2] = float("inf")
    lse = q.head_cross_entropy_fwd(X, W, t)[1]
    dW = q.head_cross_entropy_dW(X, W, t, lse, weight)
    assert torch.isinf(dW[t[2]]).all() and (dW[t[2]] < 0).all()
    weight[2] = 0
    dW = q.head_cross_entropy_dW(X, W, t, lse, weight)
    assert torch.isinf(dW[t[1]]).all() and not torch.isnan(dW).any()
