"""Tensors of the caller that a call writes have changed for autograd, too: what it had saved of them
raises in backward() instead of going into a gradient."""

import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _randn(*s, dtype=BF16):
    return torch.randn(*s, generator=torch.Generator().manual_seed(len(s))).to(dtype).to(DEV)


def _saved(t):
    """Autograd holds t for the gradient of the product's other factor."""
    other = torch.ones_like(t, requires_grad=True)
    return (other * t).sum()


@pytest.mark.parametrize("dtype", [BF16, torch.float16, torch.float32])
@pytest.mark.parametrize("max_norm", [0.1, float("inf")])
def test_clipping_in_place(dtype, max_norm):
    grads = [_randn(40, 30, dtype=dtype), _randn(7, dtype=dtype)]
    loss = [_saved(t) for t in grads]
    before = [t._version for t in grads]
    q.grad_norm(grads)
    assert [t._version for t in grads] == before
    q.clip_grad_norm(grads, max_norm)
    assert all(t._version > v for t, v in zip(grads, before))
    for one in loss:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            one.backward()


def test_clipping_into_other_tensors():
    grads = [_randn(40, 30), _randn(7)]
    outs = [torch.zeros_like(t) for t in grads]
    kept, lost = [_saved(t) for t in grads], [_saved(t) for t in outs]
    q.clip_grad_norm(grads, 0.1, out=outs)
    for one in kept:
        one.backward()
    for one in lost:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            one.backward()


def test_clipping_inference_tensors():
    """They have no version; others beside them keep theirs."""
    plain = [_randn(40, 30), _randn(7)]
    want = [torch.empty_like(t) for t in plain]
    norm = q.clip_grad_norm(plain, 0.1, out=want)
    with torch.inference_mode():
        grads = [_randn(40, 30), plain[1]]
        before = plain[1]._version
        assert torch.equal(q.clip_grad_norm(grads, 0.1), norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    assert plain[1]._version > before


@pytest.mark.parametrize("M", [9, 80])
def test_outputs_of_the_adapters(M):
    n, N, K, r = 3, 72, 128, 8
    w = q.NF4Weight.quantize(_randn(N, K, dtype=torch.float32))
    args = (w, _randn(n, r, K), _randn(n, N, r), torch.ones(n, device=DEV), torch.zeros(M, dtype=torch.int64, device=DEV))
    X, dY = _randn(M, K), _randn(M, N)
    outs = [torch.empty(s, dtype=BF16, device=DEV) for s in ((M, N), (M, r), (M, K), (n, r, K), (n, N, r))]
    before = [t._version for t in outs]
    q.adapter_linear_fwd(X, *args, out=outs[0], T_out=outs[1])
    assert [t._version for t in outs] == [before[0] + 1, before[1] + 1] + before[2:]
    q.adapter_linear_bwd(dY, X, None, *args, dX_out=outs[2], dA_out=outs[3], dB_out=outs[4])
    assert [t._version for t in outs] == [v + 1 for v in before]
    again = q.adapter_linear_bwd(dY, X, None, *args, need_dA=False, dA_out=outs[3])
    assert again[1] is None and outs[3]._version == before[3] + 1


@pytest.mark.parametrize("M", [9, 80])
def test_outputs_of_the_head(M):
    X, W, t = _randn(M, 64), _randn(300, 64), torch.arange(M, device=DEV)
    want = q.head_cross_entropy(X, W, t)
    loss = _saved(X)
    X2 = X.clone()
    kept = _saved(X2)
    q.head_cross_entropy(X2, W, t, dX_out=torch.empty_like(X))
    kept.backward()
    assert torch.equal(q.head_cross_entropy(X, W, t, dX_out=X)[2], want[2])       # over the hidden states themselves
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    dW = torch.empty_like(W)
    v = dW._version
    q.head_cross_entropy_dW(X2, W, t, want[1], dW_out=dW)
    assert dW._version == v + 1
