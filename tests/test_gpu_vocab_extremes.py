"""Vocabulary losses where the logits are large or masked by finite values of
any size: no finite row gives a NaN.

The bounds are those of test_gpu_vocab.  Large logits change nothing in them:
where z c leaves the range in which one fused multiply-add keeps t, the
kernels take z - a (one rounding, 2^-24 of |t|) times c (another), within the
2^-23 |t| counted there.  Teachers' logits are all 0 here, so q = 1 / K up to
two roundings and the loss of words far below the maximum stays within 2^-22
of itself."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from tests.gpu_util import DEV
from tests.test_gpu_vocab import (BF16, FP16, FP32, _check_distill, _check_logprobs, _check_logprobs_grad, _host64, _logits,
                                  _rows)

pytestmark = pytest.mark.gpu

# one workgroup a row (256, 512 and 1024 threads), and rows in slices
SIZES = [(FP32, 3001), (BF16, 3001), (FP16, 3001), (BF16, 32000), (FP32, 50001), (BF16, 131072)]
MASKS = {FP32: (-1e5, -1e9, -1e10, -1e12, -1e20, -1e30, -1e37, -3.3e38), FP16: (-30000.0, -50000.0, -65504.0)}
MASKS[BF16] = MASKS[FP32]


def _all_of(z, temperature=1.0, top=5):
    """Every operator on z against the oracle, and no NaN among the numbers."""
    M, V = z.shape
    target = torch.from_numpy(np.random.default_rng(V).integers(0, V, M)).to(DEV)
    r = _check_logprobs(z, target, top)
    d = _check_logprobs_grad(z, target, r, 3)
    idx = np.stack([np.random.default_rng(m).permutation(V)[:8] for m in range(M)]).astype(np.int64)
    loss, dd = _check_distill(z, idx, np.zeros((M, 8), np.float32), temperature, 5)
    for v in (r.logprob, r.entropy, r.lse, r.top_logprob, d, loss, dd):
        assert not torch.isnan(v).any()


@pytest.mark.parametrize("dtype,V", SIZES)
def test_masks_of_any_finite_value(dtype, V):
    """Whole rows, most of a row, and whole slices of a row at one value."""
    for k, low in enumerate(MASKS[dtype]):
        z = _logits(6, V, V + k, masked=False)
        z[0] = low
        z[1, 7:] = low
        z[2, : V - 50] = low
        z[3, V // 5 : 4 * V // 5] = low
        z[4] = -low                               # large and positive, all words alike
        _all_of(_rows(z, dtype, V), top=(5, 64)[k % 2])


def test_masked_slices_of_many_rows():
    """The row is cut because there are alternatives and many rows."""
    z = _logits(300, 50001, 11, masked=False)
    z[:100, 9000:30000] = -1e10
    z[100:200, 40000:] = -1e30
    z[200:250] = -1e12
    _all_of(_rows(z, FP32, 50048), top=64)


@pytest.mark.parametrize("V", [3001, 50001])
def test_rows_far_from_zero(V):
    """The same row shifted, over both forms of the exponent and their border
    (|a| log2(e) = 65536), and as far as fp32 still tells words apart."""
    shifts = (0.0, 1e4, 4.53e4, 4.55e4, 1e5, 1e6, -1e4, -4.55e4, -1e6, 3e7)
    z = _logits(len(shifts), V, 2, masked=False) + np.array(shifts)[:, None]
    _all_of(_rows(z, FP32, V))


@pytest.mark.parametrize("dtype,V", [(FP32, 3001), (BF16, 32000), (FP32, 50001)])
@pytest.mark.parametrize("temperature", [1e-3, 1e-6, 1e-9, 1e6])
def test_extreme_temperatures(dtype, V, temperature):
    """z / temperature of any size; equal maxima share the probability.  Whole
    logits: a p is a share of 1 or, over a small temperature, below 2^-149."""
    z = np.round(_logits(4, V, 7, masked=False))
    z[1, 5 :: V // 7] = 40.0
    z[2] = -3.0
    zd = _rows(z, dtype, V)
    idx = np.stack([np.random.default_rng(m).permutation(V)[:8] for m in range(4)]).astype(np.int64)
    loss, d = _check_distill(zd, idx, np.zeros((4, 8), np.float32), temperature, 6)
    assert not torch.isnan(loss).any() and not torch.isnan(d).any()
