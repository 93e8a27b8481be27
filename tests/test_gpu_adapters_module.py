"""AdapterLinear as a module: its defaults, and casts of the whole module."""

import copy

import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
ALPHA = [8.0, 4.0, 2.6]                 # 2.6 / 8 is no bfloat16


def _layer(**k):
    g = torch.Generator().manual_seed(1)
    return q.AdapterLinear((torch.randn(72, 128, generator=g) * 0.1).to(DEV), 3, 8, ALPHA, **k), g


@pytest.mark.parametrize("cast", [lambda m: m.to(BF16), lambda m: m.bfloat16(), lambda m: m.to(DEV, BF16), lambda m: copy.deepcopy(m).bfloat16(),
                                  lambda m: torch.nn.Sequential(m).to(dtype=BF16)[0], lambda m: m.half().bfloat16()])
def test_a_cast_of_the_module_keeps_the_scales(cast):
    lin, g = _layer(lora_B=torch.ones(3, 72, 8, dtype=BF16, device=DEV))
    x = torch.randn(70, 128, generator=g).to(BF16).to(DEV)
    idx = torch.randint(-1, 3, (70,), generator=g).to(DEV)
    lin.lora_A.data.copy_((torch.randint(-4, 5, lin.lora_A.shape, generator=g) / 16.0))   # the same in fp16
    want, scale = lin(x, idx), lin.scale.clone()
    lin = cast(lin)
    assert lin.scale.dtype == torch.float32 and torch.equal(lin.scale, scale)
    assert torch.equal(lin(x, idx), want)
    assert torch.equal(lin.state_dict()["scale"], scale)


def test_state_of_a_cast_module_loads():
    lin, _ = _layer()
    state = {k: v.clone() for k, v in lin.state_dict().items()}
    other, _ = _layer()
    other.scale.zero_()
    other.bfloat16().load_state_dict(state)
    assert torch.equal(other.scale, lin.scale) and other.scale.dtype == torch.float32


@pytest.mark.parametrize("M", [5, 90])
def test_a_layer_without_given_pairs_learns(M):
    """At the start the output is the base's alone, and a step's gradients move it."""
    lin, g = _layer()
    x = torch.randn(M, 128, generator=g).to(BF16).to(DEV)
    idx = (torch.arange(M) % 2).to(DEV)                  # adapter 2 has no token
    with torch.no_grad():
        assert torch.equal(lin(x, idx), lin(x, torch.full_like(idx, -1)))
    lin(x, idx).backward(torch.randn(M, 72, generator=g).to(BF16).to(DEV))
    assert lin.lora_B.grad[:2].flatten(1).any(1).all() and not lin.lora_B.grad[2].any()
    bound = 128 ** -0.5
    assert float(lin.lora_A.abs().max()) <= bound * (1 + 2.0 ** -8) and float(lin.lora_A.float().std()) > 0.4 * bound
    assert lin.lora_A.dtype == BF16 and not torch.equal(lin.lora_A[0], lin.lora_A[1])
