"""Host-side checks of the MX4 and vocabulary entry points: size queries, and
bad arguments rejected before anything is launched (no call reaches the GPU)."""

import ctypes

import pytest

import bit_nf4_quantized_absmax_amd as q
from bit_nf4_quantized_absmax_amd import _capi

OK, INVALID, SHAPE, WS = 0, -1, -2, -3
P = ctypes.c_void_p(0x20000)      # aligned, never dereferenced
ODD = ctypes.c_void_p(0x20001)
BIG = 1 << 40


def _mx4(rows, cols, codes=0x10000, scales=0x11000):
    return ctypes.byref(_capi.MX4ArrayStruct(codes, scales, rows, cols))


def _logits(rows=8, words=200000, type=1, pitch=None, z=0x30000):
    return ctypes.byref(_capi.LogitsStruct(z, type, rows, words, words if pitch is None else pitch))


def _teacher(count=8, temperature=1.0, index=0x40000, logit=0x50000):
    return ctypes.byref(_capi.TeacherStruct(index, logit, count, temperature))


def test_mx4_sizes():
    L = q.lib()
    c, s = ctypes.c_int64(), ctypes.c_int64()
    for rows, cols, kp in ((1, 32, 256), (7, 256, 256), (3, 288, 512), (0, 64, 256)):
        assert L.qlora_mx4_sizes(rows, cols, ctypes.byref(c), ctypes.byref(s)) == OK
        assert (c.value, s.value) == (rows * kp // 2, rows * kp // 32)
    assert L.qlora_mx4_sizes(1, 33, None, None) == SHAPE
    assert L.qlora_mx4_sizes(1, 0, None, None) == INVALID
    assert L.qlora_mx4_sizes(-1, 32, None, None) == INVALID
    assert L.qlora_mx4_sizes(1, (1 << 24) + 32, None, None) == SHAPE


def test_workspace_queries():
    L = q.lib()
    size = L.qlora_mx4_linear_workspace_bytes
    for M in (1, 16, 64, 65, 2047, 2048, 8192):
        # X in MX4 at least: 17 bytes a block
        assert size(M, 4096, 4096, 64, 0) >= M * 4096 * 17 // 32
        assert size(M, 4096, 4096, 0, 0) >= M * 4096 * 17 // 32
        assert size(M, 4096, 4096, 64, 1) >= 4096 * 4096 * 2
    assert size(100, 256, 8192, 0, 0) >= 100 * 8192 * 17 // 32 + 2 * 2 * 128 * 128 * 4      # two tiles in two parts or more
    for bad in ((0, 64, 64, 8, 0), (4, 64, 48, 8, 0), (4, 64, 64, 129, 0), (4, 64, 64, -1, 0), (4, 64, 64, 0, 1),
                (4, 64, 96, 8, 1), (4, 60, 64, 8, 1), (-1, 64, 64, 8, 0)):
        assert size(*bad) == 0, bad
    v = L.qlora_vocab_workspace_bytes
    assert v(1, 4, 1000, 0) == 0 and v(1, 4, 200000, 0) > 0
    assert v(1, 4, 200000, 64) >= v(1, 4, 200000, 0) + 4 * 64 * 8
    for bad in ((3, 4, 200000, 0), (-1, 4, 200000, 0), (1, 0, 200000, 0), (1, 4, 0, 0), (1, 4, 200000, 65), (1, 4, 200000, -1),
                (1, 4, 7, 8), (1, 4, 1 << 31, 0)):
        assert v(*bad) == 0, bad


def test_codec_refusals():
    L = q.lib()
    f = L.qlora_mx4_quantize
    assert f(None, 1, _mx4(4, 64), None) == INVALID
    assert f(ODD, 1, _mx4(4, 64), None) == INVALID
    assert f(P, 3, _mx4(4, 64), None) == INVALID
    assert f(P, -1, _mx4(4, 64), None) == INVALID
    assert f(P, 1, None, None) == INVALID
    assert f(P, 1, _mx4(4, 64, codes=0), None) == INVALID
    assert f(P, 1, _mx4(4, 64, scales=0x11001), None) == INVALID
    assert f(P, 1, _mx4(4, 40), None) == SHAPE
    assert f(P, 1, _mx4(0, 64), None) == OK                     # no rows: nothing to do
    assert L.qlora_mx4_dequantize(_mx4(4, 64), None, None) == INVALID
    assert L.qlora_mx4_dequantize(None, P, None) == INVALID
    assert L.qlora_mx4_dequantize(_mx4(0, 64), None, None) == OK


def test_product_refusals():
    L = q.lib()
    f = L.qlora_mx4_matmul
    x, w = _mx4(4, 64), _mx4(8, 64)
    assert f(None, w, None, None, 0, P, None) == INVALID
    assert f(x, None, None, None, 0, P, None) == INVALID
    assert f(x, _mx4(8, 96), None, None, 0, P, None) == INVALID     # other contraction
    assert f(x, _mx4(0, 64), None, None, 0, P, None) == INVALID
    assert f(x, w, None, None, 0, None, None) == INVALID
    assert f(x, w, None, None, 0, ODD, None) == INVALID
    assert f(x, w, P, None, 8, P, None) == INVALID
    assert f(x, w, None, P, 8, P, None) == INVALID
    assert f(x, w, P, P, 129, P, None) == SHAPE
    assert f(_mx4(0, 64), w, None, None, 0, None, None) == OK


def test_linear_refusals():
    L = q.lib()
    fwd, bwd = L.qlora_mx4_linear_fwd, L.qlora_mx4_linear_bwd
    w = _mx4(64, 64)
    good = lambda **k: [k.get(n, d) for n, d in (("X", P), ("M", 4), ("W", w), ("A", P), ("B", P), ("r", 8), ("scale", 1.0),
                                                  ("Y", P), ("T", P), ("ws", P), ("bytes", BIG), ("stream", None))]
    for bad, want in (({"X": None}, INVALID), ({"Y": None}, INVALID), ({"W": None}, INVALID), ({"A": None}, INVALID),
                      ({"B": ODD}, INVALID), ({"T": ODD}, INVALID), ({"scale": float("nan")}, INVALID), ({"M": -1}, INVALID),
                      ({"r": 129}, SHAPE), ({"W": _mx4(64, 72)}, SHAPE), ({"M": 1 << 31}, SHAPE), ({"ws": None}, WS),
                      ({"ws": ODD}, WS), ({"bytes": 16}, WS)):
        assert fwd(*good(**bad)) == want, bad
    assert fwd(*good(M=0, X=None, Y=None, ws=None, bytes=0)) == OK
    good = lambda **k: [k.get(n, d) for n, d in (("dY", P), ("X", P), ("T", P), ("M", 4), ("W", w), ("A", P), ("B", P), ("r", 8),
                                                  ("scale", 1.0), ("dX", P), ("dA", P), ("dB", P), ("ws", P), ("bytes", BIG),
                                                  ("stream", None))]
    for bad, want in (({"dY": None}, INVALID), ({"X": ODD}, INVALID), ({"A": None}, INVALID), ({"dX": ODD}, INVALID),
                      ({"dA": ODD}, INVALID), ({"dB": ODD}, INVALID), ({"scale": float("inf")}, INVALID), ({"r": 0}, SHAPE),
                      ({"W": _mx4(64, 96)}, SHAPE), ({"W": _mx4(72, 64)}, SHAPE), ({"ws": None}, WS), ({"bytes": 64}, WS)):
        assert bwd(*good(**bad)) == want, bad
    assert bwd(*good(M=0, dY=None, X=None, ws=None, bytes=0)) == OK


def test_vocabulary_refusals():
    L = q.lib()
    f = L.qlora_token_logprobs
    good = lambda **k: [k.get(n, d) for n, d in (("l", _logits()), ("t", P), ("top", 4), ("lp", P), ("h", P), ("lse", P), ("tl", P),
                                                  ("ti", P), ("ws", P), ("bytes", BIG), ("stream", None))]
    for bad, want in (({"l": None}, INVALID), ({"l": _logits(type=3)}, INVALID), ({"l": _logits(z=0)}, INVALID),
                      ({"l": _logits(z=0x30001)}, INVALID), ({"l": _logits(type=0, z=0x30002)}, INVALID),
                      ({"l": _logits(pitch=199999)}, INVALID), ({"l": _logits(words=0)}, INVALID), ({"l": _logits(rows=-1)}, INVALID),
                      ({"l": _logits(words=1 << 31)}, SHAPE), ({"t": None}, INVALID), ({"lp": None}, INVALID), ({"h": ODD}, INVALID),
                      ({"lse": None}, INVALID), ({"tl": None}, INVALID), ({"ti": ODD}, INVALID), ({"top": 65}, SHAPE),
                      ({"top": -1}, SHAPE), ({"l": _logits(words=3)}, SHAPE), ({"ws": None}, WS), ({"bytes": 8}, WS)):
        assert f(*good(**bad)) == want, bad
    assert f(*good(l=_logits(rows=0, z=0), t=None, lp=None, h=None, lse=None, tl=None, ti=None, ws=None, bytes=0)) == OK
    f = L.qlora_token_logprobs_bwd
    good = lambda **k: [k.get(n, d) for n, d in (("l", _logits()), ("t", P), ("lse", P), ("h", P), ("gl", P), ("gh", None), ("dz", P),
                                                  ("pitch", 200000), ("stream", None))]
    for bad in ({"t": None}, {"lse": ODD}, {"h": None}, {"gl": ODD}, {"gh": ODD}, {"dz": None}, {"dz": ODD}, {"pitch": 100}):
        assert f(*good(**bad)) == INVALID, bad


@pytest.mark.parametrize("which", ["fwd", "bwd", "both"])
def test_distillation_refusals(which):
    L = q.lib()

    def call(l=_logits(), t=_teacher(), loss=P, lse=P, w=None, dz=P, pitch=200000, ws=P, bytes=BIG):
        if which == "fwd":
            return L.qlora_distill_fwd(l, t, loss, lse, ws, bytes, None)
        if which == "bwd":
            return L.qlora_distill_bwd(l, t, lse, w, dz, pitch, None)
        return L.qlora_distill(l, t, w, loss, lse, dz, pitch, ws, bytes, None)

    nan, inf = float("nan"), float("inf")
    for bad, want in (({"l": None}, INVALID), ({"t": None}, INVALID), ({"l": _logits(pitch=5)}, INVALID), ({"lse": None}, INVALID),
                      ({"t": _teacher(index=0)}, INVALID), ({"t": _teacher(logit=0x50002)}, INVALID),
                      ({"t": _teacher(count=0)}, SHAPE), ({"t": _teacher(count=257)}, SHAPE),
                      ({"t": _teacher(temperature=0.0)}, INVALID), ({"t": _teacher(temperature=-1.0)}, INVALID),
                      ({"t": _teacher(temperature=nan)}, INVALID), ({"t": _teacher(temperature=inf)}, INVALID),
                      ({"t": _teacher(temperature=1e-45)}, INVALID)):
        assert call(**bad) == want, bad
    if which != "bwd":
        assert call(loss=None) == INVALID
        assert call(ws=None) == WS and call(bytes=4) == WS
    if which != "fwd":
        assert call(w=ODD) == INVALID and call(dz=None) == INVALID and call(pitch=1) == INVALID
