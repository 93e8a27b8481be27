"""Sizes at the limits of the MX4 entry points, on the host: what a launch
cannot count is refused (no call reaches the GPU: the ones that pass the size
checks lack an argument)."""

import ctypes

import bit_nf4_quantized_absmax_amd as q
from bit_nf4_quantized_absmax_amd import _capi

INVALID, SHAPE, WS = -1, -2, -3
P = ctypes.c_void_p(0x20000)      # aligned, never dereferenced
GROUPS = (1 << 24) - 1            # workgroups of 256 threads in 2^32 - 1


def _mx4(rows, cols):
    return ctypes.byref(_capi.MX4ArrayStruct(0x10000, 0x11000, rows, cols))


def test_codec_past_a_launch():
    quantize, dequantize = q.lib().qlora_mx4_quantize, q.lib().qlora_mx4_dequantize
    for slabs in (1, 3, 43):
        most = GROUPS // slabs * 8
        for cols in (256 * slabs, 256 * slabs - 224):
            assert quantize(None, 1, _mx4(most, cols), None) == INVALID
            assert quantize(P, 1, _mx4(most + 1, cols), None) == SHAPE
            assert dequantize(_mx4(2 * most, cols), None, None) == INVALID
            assert dequantize(_mx4(GROUPS // slabs * 16 + 1, cols), P, None) == SHAPE
    assert quantize(P, 1, _mx4((1 << 31) - 1, 1 << 24), None) == SHAPE
    assert q.lib().qlora_mx4_sizes(1 << 28, 256, None, None) == 0      # a size is known all the same


def test_layer_and_product_past_a_launch():
    L = q.lib()
    most = GROUPS * 8
    fwd = lambda M, w: L.qlora_mx4_linear_fwd(P, M, w, None, None, 0, 1.0, P, None, None, 0, None)
    assert fwd(most, _mx4(64, 256)) == WS and fwd(most + 1, _mx4(64, 256)) == SHAPE
    size = L.qlora_mx4_linear_workspace_bytes
    assert size(most, 64, 256, 0, 0) > 0 and size(most + 1, 64, 256, 0, 0) == 0
    wide = ((1 << 23) - 1) * 16     # W's rows, 16 to a workgroup of 512 threads
    for M in (1, 64):
        assert fwd(M, _mx4(wide, 32)) == WS and fwd(M, _mx4(wide + 1, 32)) == SHAPE
        assert L.qlora_mx4_matmul(_mx4(M, 32), _mx4(wide, 32), None, None, 0, None, None) == INVALID
        assert L.qlora_mx4_matmul(_mx4(M, 32), _mx4(wide + 1, 32), None, None, 0, P, None) == SHAPE
    assert fwd(65, _mx4(wide + 1, 32)) == WS
    assert L.qlora_mx4_matmul(_mx4(65, 32), _mx4(wide + 1, 32), None, None, 0, None, None) == INVALID
