"""A training step of several adapters over one frozen base, as its parts are used
together: the adapters' layer, the loss through the head, the backward pass,
each adapter's gradients clipped by its own norm; then decoding with the result."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from oracle import adapters as oad
from oracle import head as ohead
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _model(n, K, D, V, r, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*s, std):
        return (torch.randn(*s, generator=g) * std).to(DEV)

    lin = q.AdapterLinear(normal(D, K, std=K ** -0.5), n, r, [2.0 * r] * n, normal(n, r, K, std=K ** -0.5).to(BF16),
                          normal(n, D, r, std=0.05).to(BF16))
    return lin, normal(V, D, std=2 * D ** -0.5).to(BF16), g


@pytest.mark.parametrize("M", [50, 200])
def test_step_against_float64(M):
    n, K, D, V, r = 4, 128, 192, 501, 8
    lin, W, g = _model(n, K, D, V, r, seed=M)
    x = torch.randn(M, K, generator=g).to(BF16).to(DEV)
    idx = torch.randint(-1, n - 1, (M,), generator=g).to(DEV)        # the last adapter has no token
    t = torch.randint(0, V, (M,), generator=g)
    t[::5] = -100
    t = t.to(DEV)
    weight = torch.full((M,), 1.0 / M, device=DEV)
    h = lin(x, idx)
    loss = q.HeadCrossEntropyFn.apply(h, W, t)
    (loss * weight).sum().backward()
    grads = [lin.lora_A.grad, lin.lora_B.grad]
    base, s, i = _f64(lin.w.dequantize()), _f64(lin.scale), idx.cpu().numpy()
    A, B = _f64(lin.lora_A), _f64(lin.lora_B)
    # h itself is compared by its own tests; from the rounded h on
    wl, _, _, dh, _ = ohead.cross_entropy(_f64(h), _f64(W), t.cpu().numpy(), _f64(weight))
    _, dA, dB = oad.backward(dh, _f64(x), base, A, B, s, i)
    np.testing.assert_allclose(_f64(loss), wl, rtol=1e-5, atol=1e-5)
    for got, want in zip(grads, (dA, dB)):
        # dh, T or G and the result are rounded to bf16, and p before dh: four roundings, at random signs
        assert np.linalg.norm(_f64(got) - want) <= 4 * 2.0 ** -8 * np.linalg.norm(want)
    before = [v.clone() for v in grads]
    norms = q.clip_grad_norm(grads, 0.5 * float(q.grad_norm(grads, n).max()), n)
    want_n, want = oad.clip([_f64(v) for v in before], 0.5 * float(norms.max()), n)
    np.testing.assert_allclose(_f64(norms), want_n, rtol=1e-6)
    assert float(norms[n - 1]) == 0 and not any(v[n - 1].any() for v in grads)
    for got, w in zip(grads, want):
        np.testing.assert_allclose(_f64(got), w, rtol=2.0 ** -8 + 1e-6, atol=1e-38)


def test_training_the_adapters_and_decoding_with_them():
    """A few steps run, each adapter learns from its own tokens only, and a token decodes as it did within its batch."""
    n, K, D, V, r, M = 3, 128, 128, 300, 16, 300
    lin, W, g = _model(n, K, D, V, r, seed=1)
    x = torch.randn(M, K, generator=g).to(BF16).to(DEV)
    idx = torch.randint(0, 2, (M,), generator=g).to(DEV)             # adapter 2 is not used
    t = torch.randint(0, V, (M,), generator=g).to(DEV)
    held = [p.detach().clone() for p in (lin.lora_A, lin.lora_B)]
    opt = torch.optim.SGD(lin.parameters(), lr=0.5)
    for _ in range(3):
        opt.zero_grad()
        q.HeadCrossEntropyFn.apply(lin(x, idx), W, t).mean().backward()
        q.clip_grad_norm([lin.lora_A.grad, lin.lora_B.grad], 1.0, n)
        opt.step()
    assert not torch.equal(lin.lora_A[0], held[0][0]) and not torch.equal(lin.lora_B[1], held[1][1])
    assert torch.equal(lin.lora_A[2], held[0][2]) and torch.equal(lin.lora_B[2], held[1][2])
    with torch.no_grad():
        together = lin(x, idx)
        one = lin(x[7:8], idx[7:8])
    # the decoding kernels round the base weight's levels, the others their products: 2^-8 of each term, at random signs
    assert float((together[7:8] - one).float().norm()) <= 4 * 2.0 ** -8 * float(one.float().norm())
    loss, _ = q.head_cross_entropy_fwd(one, W, t[7:8])
    assert torch.isfinite(loss).all()


def test_two_streams_at_once():
    """Two calls with workspaces of their own on two streams."""
    n, K, D, V, r, M = 3, 256, 256, 2000, 16, 200
    lin, W, g = _model(n, K, D, V, r, seed=2)
    x = torch.randn(M, K, generator=g).to(BF16).to(DEV)
    idx = torch.randint(0, n, (M,), generator=g).to(DEV)
    t = torch.randint(0, V, (M,), generator=g).to(DEV)

    def both(rows):
        with torch.no_grad():
            h = lin(x[:rows], idx[:rows])
        return (h,) + q.head_cross_entropy(h, W, t[:rows])

    want = [both(M), both(40)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, rows in zip(streams, (M, 40)):
        with torch.cuda.stream(s):
            got.append([both(rows) for _ in range(4)])
    torch.cuda.synchronize()
    for runs, w in zip(got, want):
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, w))
