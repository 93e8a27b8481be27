"""Cross entropy through the output head on the GPU against the float64 oracle.

Bounds.  A logit is a sum of K products of bf16 values, exact each, in fp32: off
by at most e_z = K 2^-23 max_j sum_k |x_k| |w_jk| (0 where all sums are whole numbers
below 2^24).  e^(z - ref) adds 2^-20 (the argument, at most 16 log2(e) or small
against the largest, times 2^-24, and the hardware's exponential), so p_j is off by
e_p = 2 e_z + 2^-19 of itself, the loss by 2 e_z + 2^-19 and its own rounding.  For dX
each p_j but the target's is rounded to bf16, 2^-8 of it, and for dW each dz_mj;
words whose reference differs from their row's are brought to it by a power of two, while
the references, multiples of 64 ln 2 in fp32, are each off by 2^-23 of themselves: 2^-22 max |z|
of such a p_j for dX alone; then the gradient is rounded once, 2^-8 again; the fp32 sums between add n 2^-23 of
their terms for n terms.  What is below fp32's normal range, 2^-126, may be flushed to 0:
for dW at most 2^-126 a dz_mj and a product, for dX (e^(z - ref), against a largest of
e^-16 or more) at most 2^-126 e^16 < 2^-102 a p_j."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from oracle import head as ohead
from tests.gpu_util import DEV, Guarded, guarded_like

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
R, S = 2.0 ** -8, 2.0 ** -23


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _close(got, want, tol, name):
    got = _f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], np.broadcast_to(tol, got.shape)[bad][:4])


def _case(M, V, K, seed, whole=False, size=2.0, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    if whole:
        X = torch.randint(-3, 4, (M, K), generator=g) * (torch.rand(M, K, generator=g) < 12.0 / K)
        W = torch.randint(-2, 3, (V, K), generator=g)
    else:
        W = torch.randn(V, K, generator=g) * size * K ** -0.5
        X = torch.randn(M, K, generator=g)
    X, W = X.to(BF16), W.to(BF16)
    t = torch.randint(0, V, (M,), generator=g)
    if not whole:
        X = (X + 2.0 / size ** 2 * W[t].float() * torch.rand(M, 1, generator=g) * 2).to(BF16)
    if ignored and M > 2:
        t[torch.rand(M, generator=g) < ignored] = -100
        t[1] = V
    weight = torch.rand(M, generator=g) * 2 - 0.5
    return X.to(DEV), W.to(DEV), t.to(DEV), weight.to(DEV)


def _check(X, W, t, weight, whole=False, dW=True):
    M, K = X.shape
    V = W.shape[0]
    x, w, tt, g = _f64(X), _f64(W), t.cpu().numpy(), _f64(weight)
    loss, lse, p, dX, dWr = ohead.cross_entropy(x, w, tt, g)
    real = (tt >= 0) & (tt < V)
    ez = np.zeros(M) if whole else K * S * (np.abs(x) @ np.abs(w).T).max(1)
    ep = 2 * ez + 2.0 ** -19
    got = q.head_cross_entropy(X, W, t, weight)
    l2, lse2 = q.head_cross_entropy_fwd(X, W, t)
    for l, s in ((got[0], got[1]), (l2, lse2)):
        _close(l, loss, ep + 2.0 ** -23 * np.abs(loss), "loss")
        _close(s.double().sum(1), lse, ep + 2.0 ** -22 * np.abs(_f64(s)).sum(1), "lse")
    assert not got[0][torch.from_numpy(~real)].any()
    off = p.copy()
    off[np.arange(M), np.where(real, tt, 0)] = 0
    one = np.zeros((M, V))
    one[np.arange(M), np.where(real, tt, 0)] = real
    ag = np.abs(np.where(real, g, 0))[:, None]
    terms = ag * ((off + np.abs(p - 1) * one) @ np.abs(w))
    ez2 = 2.0 ** -22 * np.abs(np.where(real[:, None], x, 0) @ w.T).max(1)
    e = ag * ((R + (ep + ez2)[:, None] + V * S) * (off @ np.abs(w)) + (ep[:, None] + 4 * S) * ((p * one) @ np.abs(w))) + 4 * S * terms
    e = e + 2.0 ** -102 * ag * np.abs(w).sum(0) + 2.0 ** -126
    _close(got[2], dX, R * (np.abs(dX) + e) + e, "dX")
    D = torch.empty(M, K, dtype=FP32, device=DEV)
    q.head_cross_entropy(X, W, t, weight, dX_out=D)
    _close(D, dX, e + S * np.abs(dX), "dX fp32")
    assert torch.equal(D.to(BF16), got[2])
    if dW:
        d = np.abs(off + (p - 1) * one) * ag
        xa = np.where(real[:, None], np.abs(x), 0)
        e = ((R + M * S) * d + (ep[:, None] + 2.0 ** -22) * p * ag).T @ xa + 2.0 ** -126 * (2 + xa).sum(0)
        gw = q.head_cross_entropy_dW(X, W, t, got[1], weight)
        _close(gw, dWr, R * (np.abs(dWr) + e) + e, "dW")
        assert torch.equal(gw, q.head_cross_entropy_dW(X, W, t, lse2, weight)) or not torch.equal(got[1], lse2)
    return got


SHAPES = [(1, 1, 64), (1, 1000, 192), (2, 63, 64), (5, 64, 64), (16, 777, 320), (17, 65, 1088), (64, 2049, 128), (65, 256, 64),
          (100, 5003, 192), (256, 257, 64), (257, 1000, 576), (600, 300, 128)]


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("M,V,K", SHAPES)
def test_loss_and_gradients(M, V, K, whole):
    _check(*_case(M, V, K, seed=M + V, whole=whole), whole=whole)


def test_pieces_of_the_vocabulary():
    """More words than one piece at this many rows (32768)."""
    X, W, t, g = _case(4096, 40009, 64, seed=1, whole=True)
    _check(X, W, t, g, whole=True)


@pytest.mark.parametrize("M", [2, 70])
def test_a_head_past_32_bits(M):
    """More than 2^31 elements of W, all but some rows 0, so that the sums over words have few terms."""
    V, K, at = 2 ** 25 + 300, 64, 2 ** 25 + 299
    g = torch.Generator().manual_seed(M)
    some = torch.cat([torch.tensor([0, 2 ** 24, 2 ** 24 - 1, 2 ** 25 - 1, 2 ** 25, at]), torch.randint(0, V, (60,), generator=g)]).unique()
    W = torch.zeros(V, K, dtype=BF16, device=DEV)
    w = torch.randint(-2, 3, (len(some), K), generator=g).double()
    W[some.to(DEV)] = w.to(BF16).to(DEV)
    x = torch.randint(-3, 4, (M, K), generator=g) * (torch.rand(M, K, generator=g) < 0.2)
    X, x = x.to(BF16).to(DEV), x.double()
    t = torch.full((M,), at)
    z = x @ w.T                                       # the other logits are 0, as their rows are
    lse = torch.logsumexp(torch.cat([z, torch.full((M, 1), float(np.log(V - len(some))))], 1).double(), 1)
    p = torch.exp(z - lse[:, None])
    last = len(some) - 1                              # of the target
    loss, l2, dX = q.head_cross_entropy(X, W, t.to(DEV))
    ep = 2.0 ** -19
    want = (lse - z[:, last]).numpy()
    _close(loss, want, ep + S * np.abs(want), "loss")
    d = p.clone()
    d[:, last] -= 1
    e = (R + ep + 2.0 ** -22 * z.abs().max() + len(some) * S) * (d.abs() @ w.abs()) + 2.0 ** -102 * w.abs().sum(0)
    e, want = e.numpy(), (d @ w).numpy()
    _close(dX, want, R * (np.abs(want) + e) + e, "dX")
    dW = q.head_cross_entropy_dW(X, W, t.to(DEV), l2)
    one = torch.exp(-lse) @ x                         # of a word whose row is 0
    want = np.concatenate([(d.T @ x).numpy(), one.numpy()[None]])
    size = torch.cat([d.abs().T @ x.abs(), (torch.exp(-lse) @ x.abs())[None]]).numpy()
    e = (R + ep + M * S) * size + 2.0 ** -126 * (2 + x.abs().sum(0)).numpy()
    rows = [int(i) for i in some] + [next(i for i in range(2 ** 24 + 100, V) if i not in set(some.tolist()))]
    _close(dW[torch.tensor(rows, device=DEV)], want, R * (np.abs(want) + e) + e, "dW")
    W[:] = dW[rows[-1]]                               # every other row is that one
    W[some.to(DEV)] = dW[some.to(DEV)]
    assert torch.equal(W, dW)


def test_pieces_whose_largest_logits_are_far_apart():
    """Later words tower over earlier ones and the other way round, in steps past the references' 32, some only in part of a row's 64 words."""
    X, W, t, g = _case(4096, 36000, 64, seed=2, whole=True)
    X[:, 0], X[::2, 1] = 1.0, 4.0
    W[:, 0] = torch.arange(36000, device=DEV) // 1000 * 8            # up to 280
    W[:, 1] = -(torch.arange(36000, device=DEV) // 50 % 40).to(W.dtype) * 4
    t[0], t[2], t[3] = 35999, 5, 20000
    _check(X, W, t, g, whole=True, dW=False)
    W[:, 0] = W[:, 0].flip(0)
    _check(X, W, t, g, whole=True, dW=False)


@pytest.mark.parametrize("size", [1e3, 1e6, 1e30, 1e37])
def test_logits_of_any_finite_size(size):
    """One word far above all others, by far more than an exponential holds."""
    M, V, K = 70, 300, 64
    X = torch.zeros(M, K, dtype=BF16, device=DEV)
    W = torch.zeros(V, K, dtype=BF16, device=DEV)
    X[:, 0] = 1.0
    W[7, 0], W[200, 0] = size, -size
    t = torch.full((M,), 7, device=DEV)
    t[1], t[2] = 9, 200
    loss, lse, dX = q.head_cross_entropy(X, W, t)
    big = float(W[7, 0])
    want = torch.zeros(M, dtype=torch.float64)
    want[1], want[2] = big, 2 * big
    np.testing.assert_allclose(_f64(loss), want.numpy(), rtol=1e-6)
    wx = torch.zeros(M, K, dtype=torch.float64)
    wx[1, 0], wx[2, 0] = big, 2 * big
    np.testing.assert_allclose(_f64(dX), wx.numpy(), rtol=R)
    dW = _f64(q.head_cross_entropy_dW(X, W, t, lse))
    wd = np.zeros((V, K))
    wd[7, 0], wd[9, 0], wd[200, 0] = 2, -1, -1
    np.testing.assert_allclose(dW, wd, atol=1e-30)


def test_a_sure_target_keeps_its_small_gradient():
    """p_t = 1 - 1e-4: the gradient is 1e-4 of the words' weights, and still right to a rounding."""
    M, V, K = 8, 500, 64
    X, W, t, _ = _case(M, V, K, seed=5, ignored=0)
    X = torch.zeros_like(X)
    X[:, :3] = torch.tensor([4.0, 3.0, 2.0], device=DEV)
    W[:, :3] = 0
    W[t[:1], 0] = 4.0
    t = t[:1].expand(M).contiguous()
    got = _check(X, W, t, torch.ones(M, device=DEV), whole=False)
    assert 1e-6 < float(got[0][0]) < 1e-3


@pytest.mark.parametrize("M", [40, 300])
def test_rows_without_a_target_may_hold_anything(M):
    X, W, t, g = _case(M, 700, 128, seed=3)
    want = q.head_cross_entropy(X, W, t, g)
    dW = q.head_cross_entropy_dW(X, W, t, want[1], g)
    none = (t < 0) | (t >= 700)
    X2, g2 = X.clone(), g.clone()
    X2[none], g2[none] = float("nan"), float("inf")
    got = q.head_cross_entropy(X2, W, t, g2)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert not got[2][none].any()
    lse = got[1].clone()
    lse[none] = float("nan")
    assert torch.equal(q.head_cross_entropy_dW(X2, W, t, lse, g2), dW)


@pytest.mark.parametrize("M", [40, 300])
def test_nan_stays_in_its_row(M):
    X, W, t, g = _case(M, 700, 128, seed=3, ignored=0)
    t[1] = 4
    want = q.head_cross_entropy(X, W, t, g)
    X2 = X.clone()
    X2[5, 3], X2[M - 1, 0] = float("nan"), float("inf")
    got = q.head_cross_entropy(X2, W, t, g)
    ok = torch.ones(M, dtype=torch.bool, device=DEV)
    ok[5] = ok[M - 1] = False
    for a, b in zip(got, want):
        assert torch.equal(a[ok], b[ok])
    assert torch.isnan(got[0][~ok]).all() and torch.isnan(got[2][~ok]).any(1).all()


def test_no_targets_and_no_rows():
    X, W, t, g = _case(90, 300, 64, seed=4)
    t.fill_(-100)
    loss, lse, dX = q.head_cross_entropy(X, W, t, g)
    assert not loss.any() and not lse.any() and not dX.any()
    dW = torch.full_like(W, float("nan"))
    assert not q.head_cross_entropy_dW(X, W, t, lse, g, dW_out=dW).any()
    e = slice(0, 0)
    loss, lse, dX = q.head_cross_entropy(X[e], W, t[e], g[e])
    assert loss.shape == (0,) and lse.shape == (0, 2) and dX.shape == (0, 64)
    dW.fill_(float("nan"))
    assert not q.head_cross_entropy_dW(X[e], W, t[e], lse, dW_out=dW).any()


@pytest.mark.parametrize("M", [3, 64, 90])
def test_nothing_outside_the_outputs_is_written(M):
    V, K = 333, 192
    X, W, t, g = _case(M, V, K, seed=M)
    L = q.lib()
    ws = [Guarded(L.qlora_head_workspace_bytes(M, V, K, k), k) for k in range(3)]
    gx, dX = guarded_like((M, K), seed=5)
    gw, dW = guarded_like((V, K), seed=6)
    gd, D = guarded_like((M, K), FP32, seed=7)
    q.head_cross_entropy_fwd(X, W, t, workspace=ws[0].payload)
    _, lse, _ = q.head_cross_entropy(X, W, t, g, dX_out=dX, workspace=ws[1].payload)
    q.head_cross_entropy(X, W, t, g, dX_out=D, workspace=ws[1].payload)
    q.head_cross_entropy_dW(X, W, t, lse, g, dW_out=dW, workspace=ws[2].payload)
    assert all(b.intact() for b in ws + [gx, gw, gd])
    assert all(torch.isfinite(v).all() for v in (dX, D, dW))


@pytest.mark.parametrize("M,V,K", [(7, 300, 64), (130, 500, 128)])
def test_autograd(M, V, K):
    X, W, t, g = _case(M, V, K, seed=M)
    xa, wa = X.clone().requires_grad_(), W.clone().requires_grad_()
    loss = q.HeadCrossEntropyFn.apply(xa, wa, t)
    want = q.head_cross_entropy(X, W, t, g)
    assert torch.equal(loss, want[0])
    (loss * g).sum().backward()
    assert torch.equal(wa.grad, q.head_cross_entropy_dW(X, W, t, want[1], g))
    np.testing.assert_allclose(_f64(xa.grad), _f64(want[2]), rtol=2 * R, atol=1e-12)   # another order of the fp32 product by g
    xb = X.clone().requires_grad_()
    q.HeadCrossEntropyFn.apply(xb, W, t).backward(g)
    assert torch.equal(xb.grad, xa.grad)
    wb = W.clone().requires_grad_()
    q.HeadCrossEntropyFn.apply(X, wb, t).backward(g)
    assert torch.equal(wb.grad, wa.grad)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(q.HeadCrossEntropyFn.apply(xb, W, t).sum(), xb, create_graph=True)[0].sum().backward()
    assert not q.HeadCrossEntropyFn.apply(X, W, t).requires_grad
    # against differences
    x, w, tt = _f64(X), _f64(W), t.cpu().numpy()
    r = np.random.default_rng(1)
    for grad, v in ((xa.grad, r.standard_normal(x.shape)), (wa.grad, r.standard_normal(w.shape))):
        h = 1e-4
        f = [(ohead.cross_entropy(x + (s * h * v if v.shape == x.shape else 0), w + (s * h * v if v.shape == w.shape else 0), tt,
                                  _f64(g))[0] * _f64(g)).sum() for s in (1, -1)]
        got = (_f64(grad) * v).sum()
        assert abs(got - (f[0] - f[1]) / (2 * h)) <= 6 * R * np.sqrt((_f64(grad) ** 2 * v ** 2).sum()) + 1e-6


@pytest.mark.parametrize("M", [20, 300])
def test_captured_and_replayed(M):
    V, K = 1000, 128
    X, W, t, g = _case(M, V, K, seed=M)
    L = q.lib()
    ws = [torch.empty(L.qlora_head_workspace_bytes(M, V, K, k), dtype=torch.uint8, device=DEV) for k in (1, 2)]
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    held = {}

    def step():
        held["loss"], held["lse"], _ = q.head_cross_entropy(X, W, t, g, dX_out=dX, workspace=ws[0])
        q.head_cross_entropy_dW(X, W, t, held["lse"], g, dW_out=dW, workspace=ws[1])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        X2, _, t2, g2 = _case(M, V, K, seed=10 + k, ignored=0.3 * k)
        X.copy_(X2), t.copy_(t2), g.copy_(g2)
        dX.fill_(float("nan")), dW.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (held["loss"], held["lse"], dX, dW)]
        want = q.head_cross_entropy(X, W, t, g)
        want += (q.head_cross_entropy_dW(X, W, t, want[1], g),)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    X, W, t, g = _case(10, 300, 128, seed=1)
    for bad, err in (((X, W[:, :64].contiguous(), t), ValueError), ((X, W, t.int()), TypeError), ((X, W, t[:-1]), ValueError),
                     ((X.float(), W, t), TypeError), ((X, W.float(), t), TypeError), ((X.cpu(), W, t), ValueError),
                     ((X[:, :96].contiguous(), W[:, :96].contiguous(), t), q.QLoRAError), ((X, W.t(), t), ValueError),
                     ((X, W, t, g.double()), TypeError), ((X, W, t, g[:-1]), ValueError)):
        with pytest.raises(err):
            q.head_cross_entropy(*bad)
    with pytest.raises(ValueError):
        q.head_cross_entropy(X, W, t, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        q.head_cross_entropy(X, W, t, dX_out=torch.empty(10, 128, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):
        q.head_cross_entropy_dW(X, W, t, torch.zeros(10, device=DEV))
