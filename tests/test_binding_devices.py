"""Tensors in host memory raise before anything is launched: their addresses
mean nothing to a kernel (no call here reaches a GPU)."""

import pytest
import torch

import bit_nf4_quantized_absmax_amd as q

BF16 = torch.bfloat16


def _weight(rows=64, cols=128):
    n = rows * cols
    return q.NF4Weight(torch.zeros(n // 2, dtype=torch.uint8), torch.zeros(n // 64, dtype=torch.uint8),
                       torch.zeros(1), torch.zeros(1), rows, cols)


def test_nf4_weight_in_host_memory():
    w = _weight()
    with pytest.raises(ValueError):
        w.dequantize()
    with pytest.raises(ValueError):
        q.dequantize_group([w, _weight(64, 64)])
    with pytest.raises(ValueError):
        q.NF4Weight.quantize(torch.zeros(64, 128))


def test_mx4_array_in_host_memory():
    a = q.MX4Tensor.empty(8, 64, "cpu")
    x = torch.zeros(4, 64, dtype=BF16)
    for call in (a.dequantize, lambda: q.MX4Tensor.quantize(x), lambda: q.mx4_matmul(a, a), lambda: q.mx4_linear_fwd(x, a)):
        with pytest.raises(ValueError):
            call()


def test_logits_in_host_memory():
    z, t = torch.zeros(4, 50), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        q.token_logprobs(z, t)
    with pytest.raises(ValueError):
        q.distill_topk(z, torch.zeros(4, 3, dtype=torch.int64), torch.zeros(4, 3))
