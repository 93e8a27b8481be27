"""The MX4 and vocabulary operators where a training loop goes beyond one plain
step: a batch without tokens, results changed in place, a gradient of a
gradient."""

import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _dirty(*shapes):
    """Leaves freed memory of these shapes behind that holds no zeros."""
    held = [torch.full(s, float("nan"), dtype=BF16, device=DEV) for s in shapes]
    del held


def _pair(N, K, r):
    g = torch.Generator().manual_seed(N + K)
    W, A, B = torch.randn(N, K, generator=g), torch.randn(r, K, generator=g), torch.randn(N, r, generator=g)
    return q.MX4Linear(W.to(DEV), r, 8.0, A.to(BF16).to(DEV), B.to(BF16).to(DEV))


@pytest.mark.parametrize("N,K,r", [(128, 320, 8), (4096, 4096, 64)])
def test_no_tokens_have_zero_gradients(N, K, r):
    """A batch (an expert, a micro-batch) without tokens adds nothing to the adapter's gradients."""
    lin = _pair(N, K, r)
    x = torch.empty(0, K, dtype=BF16, device=DEV, requires_grad=True)
    _dirty((r, K), (N, r))
    lin(x).sum().backward()
    assert x.grad.shape == (0, K)
    assert lin.lora_A.grad.shape == (r, K) and not lin.lora_A.grad.any()
    assert lin.lora_B.grad.shape == (N, r) and not lin.lora_B.grad.any()


def test_no_tokens_into_given_gradients():
    lin = _pair(128, 320, 8)
    A, B = lin.lora_A.detach(), lin.lora_B.detach()
    x, dy = (torch.empty(0, n, dtype=BF16, device=DEV) for n in (320, 128))
    dA, dB = torch.ones_like(A), torch.ones_like(B)
    got = q.mx4_linear_bwd(dy, x, None, lin.w, A, B, 1.0, dA_out=dA, dB_out=dB)
    assert got[1] is dA and got[2] is dB and not dA.any() and not dB.any()
    got = q.mx4_linear_bwd(dy, x, None, lin.w, A, B, 1.0, need_dX=False, need_dB=False)
    assert got[0] is None and got[2] is None and not got[1].any()


def test_results_may_be_changed_in_place():
    """A loss mask applied to the log probabilities where they lie, with and without autograd."""
    g = torch.Generator().manual_seed(3)
    z = torch.randn(6, 500, generator=g).to(DEV)
    t = torch.arange(6, device=DEV)
    mask = torch.tensor([1.0, 0.0, 1.0, 1.0, 0.0, 1.0], device=DEV)
    za, zb = z.clone().requires_grad_(), z.clone().requires_grad_()
    lp, h = q.TokenLogprobsFn.apply(za, t)
    lp *= mask
    (lp.sum() + h.sum()).backward()
    lp, h = q.TokenLogprobsFn.apply(zb, t)
    ((lp * mask).sum() + h.sum()).backward()
    assert torch.equal(za.grad, zb.grad) and za.grad.any()
    r = q.token_logprobs(z, t)
    entropy = r.entropy.clone()
    coef = torch.ones(6, device=DEV, requires_grad=True)
    r.logprob.mul_(coef).sum().backward()
    assert coef.grad.any() and torch.equal(r.entropy, entropy)


def test_second_derivatives_are_refused():
    """Gradients are computed outside autograd: a gradient of one raises, it is not taken as constant."""
    g = torch.Generator().manual_seed(4)
    z = torch.randn(3, 40, generator=g).to(DEV).requires_grad_()
    lin = _pair(64, 64, 8)
    x = torch.randn(5, 64, generator=g).to(BF16).to(DEV).requires_grad_()
    idx = torch.arange(4, device=DEV).repeat(3, 1)
    val = torch.zeros(3, 4, device=DEV)
    for leaf, out in ((z, lambda: q.TokenLogprobsFn.apply(z, torch.arange(3, device=DEV))[0]),
                      (z, lambda: q.DistillTopKFn.apply(z, idx, val, 1.0)), (x, lambda: lin(x))):
        first, = torch.autograd.grad((out().float() ** 2).sum() + (leaf.float() ** 2).sum(), leaf, create_graph=True)
        assert first.any()
        with pytest.raises(RuntimeError):
            (first.float() ** 2).sum().backward()
