"""The target's own term of the head's cross entropy, from unsure to sure targets, on the
GPU against float64, each quantity held to a bound relative to itself.

Logits are whole numbers, exact in fp32, and within 128 of each other.  An exponential that
is not flushed has an argument x of at most 88: its fp32 steps (the distance to the
reference, the rest, the factor log2 e and its product) are off by 2^-24 |x| each at most,
the rest by 2^-24 of up to 66, the hardware's by 2^-23: 2^-15 of the value in all.  The sum of
the words but the target and its join of references are within 2^-14 of themselves, and so are the
loss (log1p of it) and p_t - 1 = expm1(-loss) where the target is sure; where it is not, 1 - p_t is 0.39
at least and p_t's 2^-14 are 2^-12 of it at most: D = 2^-11 bounds them all.  p_j and dz are rounded to bf16,
2^-8, gradients once more; fp32 sums of n terms add n 2^-23 of their terms.  What is below 2^-126 may be 0: for dX
that is an exponential against a largest of 2^-32 or more, 2^-94 of the other words' sum."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
R, S, D = 2.0 ** -8, 2.0 ** -23, 2.0 ** -11
ABOVE = [0, 5, 6, 7, 8, 16, 20, 30, 60, 100]      # the target's logit over the other words' largest, by group of rows
V, K = 500, 64


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _case(M, base):
    """Group k's rows name word 7 + 49 k, whose logit is base + ABOVE[k]; the other words' are base - 0 .. 8."""
    g = torch.Generator().manual_seed(M)
    n = len(ABOVE)
    word = 7 + 49 * torch.arange(n)
    X, W = torch.zeros(M, K), torch.zeros(V, K)
    W[:, 0] = base - (torch.arange(V) % 3).float()
    W[word, 0] = base - 8.0
    W[word, 1 + torch.arange(n)] = 1.0
    group = torch.arange(M) % n
    X[:, 0] = 1.0
    X[torch.arange(M), 1 + group] = torch.tensor(ABOVE).float()[group] + 8.0
    X[:, 12:36] = torch.randint(-3, 4, (M, 24), generator=g).float()      # where W is 0, for dW
    W[:, 36:] = torch.randint(-3, 4, (V, K - 36), generator=g).float()    # where X is 0, for dX
    weight = torch.rand(M, generator=g) + 0.5
    return X, W, word[group], weight, word


@pytest.mark.parametrize("base", [0, -20, 50])
@pytest.mark.parametrize("M", [10, 64, 70, 300])
def test_the_targets_term_from_unsure_to_sure(M, base):
    X, W, t, weight, word = _case(M, base)
    x, w, g = X.double().numpy(), W.double().numpy(), weight.double().numpy()
    rows = np.arange(M)
    z = x @ w.T
    zt = z[rows, t]
    e = np.exp(z - zt[:, None])
    e[rows, t] = 0.0
    total = e.sum(1)                                   # of the other words, against the target
    loss = np.log1p(total)
    off = e / (1 + total)[:, None]
    own = -total / (1 + total)                         # p_t - 1
    d = off.copy()
    d[rows, t] = own
    d *= g[:, None]
    Xd, Wd, td, gd = X.to(BF16).to(DEV), W.to(BF16).to(DEV), t.to(DEV), weight.to(DEV)
    got_loss, lse, dX = q.head_cross_entropy(Xd, Wd, td, gd)
    assert (np.abs(_f64(got_loss) - loss) <= D * loss + 2.0 ** -126).all()
    assert (np.abs(_f64(lse).sum(1) - (zt + loss)) <= D * np.minimum(loss, 1) + 2.0 ** -22 * np.abs(_f64(lse)).sum(1)).all()

    aw = np.abs(w)
    want = d @ w
    terms = g[:, None] * (off @ aw + np.abs(own)[:, None] * aw[t])
    err = g[:, None] * ((R + V * S) * (off @ aw) + 2.0 ** -94 * off.sum(1)[:, None] * aw.sum(0)) + (D + 4 * S) * terms + 2.0 ** -126
    tol = R * (np.abs(want) + err) + err
    assert (np.abs(_f64(dX) - want) <= tol).all()

    ax = np.abs(x)
    want_w = d.T @ x
    err = (R + D + M * S) * (np.abs(d).T @ ax) + 2.0 ** -126 * (2 + 2 * ax.sum(0))
    tol_w = R * (np.abs(want_w) + err) + err
    # nothing but the target's term reaches these: no gradient at all would not pass
    k = [i for i, v in enumerate(ABOVE) if v <= 60]
    assert (tol_w[word[k], 1 + np.array(k)] < 0.1 * np.abs(want_w[word[k], 1 + np.array(k)])).all()
    sure = [m for m in rows if ABOVE[m % len(ABOVE)] <= 60]
    assert (tol[sure, 1 + np.array(sure) % len(ABOVE)] < 0.1 * np.abs(want[sure, 1 + np.array(sure) % len(ABOVE)])).all()
    for pair in (lse, q.head_cross_entropy_fwd(Xd, Wd, td)[1]):
        dW = _f64(q.head_cross_entropy_dW(Xd, Wd, td, pair, gd))
        bad = ~(np.abs(dW - want_w) <= tol_w)
        assert not bad.any(), (np.argwhere(bad)[:4], dW[bad][:4], want_w[bad][:4], tol_w[bad][:4])


@pytest.mark.parametrize("M", [10, 70])
def test_autograd_of_a_sure_target(M):
    """The same term by way of backward(), one group of rows at a time."""
    X, W, t, weight, word = _case(M, 0)
    rows = torch.arange(M) % len(ABOVE) == ABOVE.index(20)
    X, t, weight = X[rows], t[rows], weight[rows]
    wa = W.to(BF16).to(DEV).requires_grad_()
    q.HeadCrossEntropyFn.apply(X.to(BF16).to(DEV), wa, t.to(DEV)).backward(weight.to(DEV))
    z = X.double() @ W.double().t()
    at = int(t[0])
    others = torch.exp(z - z[:, at:at + 1])
    others[:, at] = 0
    total = others.sum(1)
    want = float((-total / (1 + total) * weight.double() * X[:, 1 + ABOVE.index(20)].double()).sum())
    assert abs(float(wa.grad[at, 1 + ABOVE.index(20)]) - want) <= (2 * R + D + M * S) * abs(want)
