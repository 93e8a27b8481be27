"""Sizes at the limits of the vocabulary losses, on the host: what a kernel's
offsets or a launch cannot count is refused, what they can is not (no call
reaches the GPU: the ones that pass the size checks lack an argument)."""

import ctypes

import pytest

import bit_nf4_quantized_absmax_amd as q
from bit_nf4_quantized_absmax_amd import _capi

INVALID, SHAPE = -1, -2
P = ctypes.c_void_p(0x20000)      # aligned, never dereferenced
FP32, BF16, FP16 = 0, 1, 2
ROW_BYTES = (1 << 32) - (1 << 24)


def _calls(type, rows, words, top=0):
    """Status of each call on such logits, without a target, an lse or a workspace."""
    L = q.lib()
    l = ctypes.byref(_capi.LogitsStruct(0x30000, type, rows, words, words))
    t = ctypes.byref(_capi.TeacherStruct(0x40000, 0x50000, 8, 1.0))
    return {
        "logprobs": L.qlora_token_logprobs(l, None, top, P, P, P, P, P, None, 0, None),
        "logprobs_bwd": L.qlora_token_logprobs_bwd(l, None, P, P, P, P, P, words, None),
        "distill_fwd": L.qlora_distill_fwd(l, t, P, None, None, 0, None),
        "distill_bwd": L.qlora_distill_bwd(l, t, None, None, P, words, None),
        "distill": L.qlora_distill(l, t, None, P, None, P, words, None, 0, None),
    }


@pytest.mark.parametrize("type,size", [(FP32, 4), (BF16, 2), (FP16, 2)])
def test_rows_past_32_bit_offsets(type, size):
    most = ROW_BYTES // size
    assert set(_calls(type, 1, most).values()) == {INVALID}
    assert q.lib().qlora_vocab_workspace_bytes(type, 1, most, 64) > 0
    for words in (most + 1, (1 << 32) // size, (1 << 32) // size + 64, (1 << 31) - 65, 1 << 40):
        if words > most:
            assert set(_calls(type, 1, words).values()) == {SHAPE}, words
            assert q.lib().qlora_vocab_workspace_bytes(type, 1, words, 0) == 0


@pytest.mark.parametrize("type", [FP32, BF16, FP16])
def test_rows_past_a_launch(type):
    """A launch holds 2^32 - 1 threads, 256 a row at least."""
    query = q.lib().qlora_vocab_workspace_bytes
    assert set(_calls(type, (1 << 24) - 1, 1000).values()) == {INVALID}
    assert set(_calls(type, 1 << 24, 1000).values()) == {SHAPE}
    assert set(_calls(type, 1 << 40, 1000).values()) == {SHAPE}
    assert set(_calls(type, (1 << 63) - 1, 1).values()) == {SHAPE}
    # rows in slices: as many workgroups of 256 threads as their 2048 vectors fill
    n = 4 if type == FP32 else 8
    slices = -(-(200000 // n) // 2048)
    most = ((1 << 32) - 1) // (256 * slices)
    assert query(type, most // 2, 200000, 64) > 0
    assert query(type, most + 1, 200000, 64) == 0 and query(type, 1 << 30, 200000, 0) == 0
    assert _calls(type, most + 1, 200000, 64)["logprobs"] == SHAPE
    # a gradient workgroup takes 1024 vectors; the distillation's takes a whole row where there are many
    chunks = -(-200000 // n // 1024)
    most = ((1 << 32) - 1) // (256 * chunks)
    got = _calls(type, most + 1, 200000)
    assert got["logprobs_bwd"] == SHAPE and got["distill_bwd"] == INVALID
