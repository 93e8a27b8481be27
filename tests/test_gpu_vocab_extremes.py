"""Vocabulary losses where the logits are large, masked by finite values of any
size, or not numbers: no finite row gives a NaN, and every alternative is a
word of its row.

The bounds are those of test_gpu_vocab.  Large logits change nothing in them:
where z c leaves the range in which one fused multiply-add keeps t, the
kernels take z - a (one rounding, 2^-24 of |t|) times c (another), within the
2^-23 |t| counted there.  Teachers' logits are all 0 here, so q = 1 / K up to
two roundings and the loss of words far below the maximum stays within 2^-22
of itself."""

import ctypes

import numpy as np
import pytest
import torch

import bit_nf4_quantized_absmax_amd as q
from bit_nf4_quantized_absmax_amd._capi import LogitsStruct
from tests.gpu_util import DEV, Guarded
from tests.test_gpu_vocab import (BF16, FP16, FP32, _check_distill, _check_logprobs, _check_logprobs_grad, _close, _host64,
                                  _logits, _rows)

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


def _raw_alternatives(z, top):
    """qlora_token_logprobs into buffers that hold -7: (logprob, top_logprob, top_index)."""
    M, V = z.shape
    st = LogitsStruct(z.data_ptr(), {FP32: 0, BF16: 1, FP16: 2}[z.dtype], M, V, z.stride(0))
    lp, h, lse, tl = (torch.full(s, -7.0, device=DEV) for s in ((M,), (M,), (M, 2), (M, top)))
    ti = torch.full((M, top), -7, dtype=torch.int64, device=DEV)
    t = torch.zeros(M, dtype=torch.int64, device=DEV)
    need = q.lib().qlora_vocab_workspace_bytes(st.type, M, V, top)
    ws = Guarded(max(need, 16))
    assert q.lib().qlora_token_logprobs(ctypes.byref(st), t.data_ptr(), top, lp.data_ptr(), h.data_ptr(), lse.data_ptr(),
                                        tl.data_ptr(), ti.data_ptr(), ws.payload.data_ptr(), need, 0) == 0
    torch.cuda.synchronize()
    assert ws.intact()
    return lp, tl, ti


@pytest.mark.parametrize("dtype,V", [(FP32, 9), (BF16, 64), (FP16, 700), (FP32, 9000), (BF16, 40000), (FP32, 60001), (BF16, 131073)])
def test_alternatives_of_rows_with_nan_are_words_of_the_row(dtype, V):
    """NaN of either sign, quiet or signalling: every place is filled, with different words of the row."""
    bits, neg, quiet, loud = {FP32: (torch.int32, -(1 << 31), 0x7FC00000, 0x7F800001), BF16: (torch.int16, -(1 << 15), 0x7FC0, 0x7F81),
                              FP16: (torch.int16, -(1 << 15), 0x7E00, 0x7C01)}[dtype]
    z = _logits(12, V, 3, masked=False)
    z[10], z[11, V // 2:] = -np.inf, -np.inf
    zd = _rows(z, dtype, V)
    raw = zd.view(bits)
    raw[0], raw[1], raw[2], raw[3] = quiet, quiet + neg, loud, loud + neg
    raw[4, V // 3], raw[5, V // 3], raw[6, 1::2], raw[7, 1:] = quiet + neg, loud, quiet + neg, quiet + neg
    raw[8, ::3], raw[9, V - 1], raw[10, :1] = loud + neg, quiet, quiet + neg
    zeros = torch.zeros(12, dtype=torch.int64, device=DEV)
    for top in sorted({1, min(7, V), min(64, V)}):
        lp, tl, ti = _raw_alternatives(zd, top)
        want = [True] * 11 + [False]
        assert torch.isnan(lp).tolist() == want and torch.isnan(tl).all(1).tolist() == want
        assert ((ti >= 0) & (ti < V)).all(), top
        assert all(row.unique().numel() == top for row in ti), top
        alone = _check_logprobs(zd[11:], zeros[:1], top)               # a row without one is as it is by itself
        assert torch.equal(alone.top_index[0], ti[11])                 # (its sums too, where M cuts it alike)
        _close(_host64(tl[11]), _host64(alone.top_logprob[0]), 2 * (1e-5 + 2.0 ** -23 * np.abs(_host64(tl[11]))), "top")
