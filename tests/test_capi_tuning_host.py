"""Host-side checks of the entry points for many adapters, the head's cross entropy
and the gradient norm: size queries, and bad arguments rejected before anything
is launched (no call reaches the GPU)."""

import ctypes
import struct

import bit_nf4_quantized_absmax_amd as q
from bit_nf4_quantized_absmax_amd import _capi

OK, INVALID, SHAPE, WS = 0, -1, -2, -3
P = ctypes.c_void_p(0x20000)      # aligned, never dereferenced
ODD = ctypes.c_void_p(0x20001)
BIG = 1 << 44


def _weight(rows=64, cols=128, packed=0x10000, qtype=0):
    return ctypes.byref(_capi.NF4WeightStruct(packed, 0x11000, 0x12000, 0x13000, rows, cols, qtype))


def _set(n=4, r=8, A=0x30000, B=0x31000, scale=0x32000, index=0x33000):
    return ctypes.byref(_capi.AdaptersStruct(A, B, scale, index, n, r))


def test_adapter_sizes():
    size = q.lib().qlora_adapter_linear_workspace_bytes
    for M in (1, 16, 64, 65, 512, 8192):
        for n, r in ((1, 8), (64, 64), (1023, 128)):
            assert size(M, 4096, 4096, n, r, 0) >= M * r * 2
            assert size(M, 4096, 4096, n, r, 1) >= 4096 * 4096 * 2 + 2 * n * r * 4096 * 2
    assert size(65, 4096, 4096, 1, 8, 0) >= 4096 * 4096 * 2
    assert size(100, 72, 128, 2, 8, 1) >= 100 * 128 * 2                      # rows of dY filled up to 128
    for bad in ((0, 64, 128, 4, 8, 0), (-1, 64, 128, 4, 8, 0), (4, 60, 128, 4, 8, 0), (4, 64, 96, 4, 8, 0), (4, 64, 128, 0, 8, 0),
                (4, 64, 128, 1024, 8, 0), (4, 64, 128, 4, 12, 0), (4, 64, 128, 4, 136, 0), (4, 64, 128, 4, 0, 0), (1 << 31, 64, 128, 4, 8, 0),
                (4, 1 << 20, 1 << 11, 4, 8, 0), (4, 8, 1 << 24, 4, 128, 0), (4, 1 << 24, 64, 4, 128, 1)):
        assert size(*bad) == 0, bad


def test_adapter_refusals():
    L = q.lib()
    names = ("X", "M", "W", "ad", "Y", "T", "ws", "bytes", "stream")
    good = dict(X=P, M=4, W=_weight(), ad=_set(), Y=P, T=P, ws=P, bytes=BIG, stream=None)

    def fwd(**k):
        return L.qlora_adapter_linear_fwd(*[{**good, **k}[n] for n in names])

    for bad, want in (({"X": None}, INVALID), ({"X": ODD}, INVALID), ({"Y": None}, INVALID), ({"T": ODD}, INVALID), ({"W": None}, INVALID),
                      ({"ad": None}, INVALID), ({"M": -1}, INVALID), ({"W": _weight(packed=0)}, INVALID), ({"W": _weight(qtype=3)}, INVALID),
                      ({"W": _weight(rows=0)}, INVALID), ({"ad": _set(A=0)}, INVALID), ({"ad": _set(B=0x31008)}, INVALID),
                      ({"ad": _set(scale=0)}, INVALID), ({"ad": _set(index=0)}, INVALID), ({"ad": _set(index=0x33004)}, INVALID),
                      ({"ad": _set(n=0)}, INVALID), ({"ad": _set(n=1024)}, SHAPE), ({"ad": _set(r=4)}, SHAPE), ({"ad": _set(r=136)}, SHAPE),
                      ({"W": _weight(cols=96)}, SHAPE), ({"W": _weight(rows=60)}, SHAPE),
                      ({"W": _weight(rows=8, cols=1 << 24), "ad": _set(r=128)}, SHAPE), ({"M": 1 << 31}, SHAPE), ({"ws": None}, WS),
                      ({"ws": ODD}, WS), ({"bytes": 64}, WS), ({"M": 100, "bytes": 4096}, WS)):
        assert fwd(**bad) == want, bad
    assert fwd(M=0, X=None, Y=None, T=None, ws=None, bytes=0, ad=_set(index=0)) == OK
    names_b = ("dY", "X", "T", "M", "W", "ad", "dX", "dA", "dB", "ws", "bytes", "stream")
    good_b = dict(dY=P, X=P, T=P, M=4, W=_weight(), ad=_set(), dX=P, dA=P, dB=P, ws=P, bytes=BIG, stream=None)

    def bwd(**k):
        return L.qlora_adapter_linear_bwd(*[{**good_b, **k}[n] for n in names_b])

    for bad, want in (({"dY": None}, INVALID), ({"X": ODD}, INVALID), ({"T": ODD}, INVALID), ({"dX": ODD}, INVALID), ({"dA": ODD}, INVALID),
                      ({"dB": ODD}, INVALID), ({"ad": _set(r=20)}, SHAPE), ({"ws": None}, WS), ({"bytes": 256}, WS)):
        assert bwd(**bad) == want, bad
    assert bwd(M=0, dY=None, X=None, ws=None, bytes=0) == OK
    assert bwd(dX=None, dA=None, dB=None, ws=None, bytes=0) == OK        # nothing asked for


def test_head_sizes():
    size = q.lib().qlora_head_workspace_bytes
    for M in (1, 64, 65, 8192):
        assert 0 < size(M, 32000, 4096, 0) < size(M, 32000, 4096, 1)
        assert size(M, 32000, 4096, 2) >= M * 4096 * 2
    assert size(1 << 20, 131072, 64, 1) < 1 << 31                        # pieces, not logits
    for bad in ((0, 100, 64, 0), (-1, 100, 64, 0), (4, 0, 64, 0), (4, 100, 96, 0), (4, 100, 0, 0), (4, 100, 64, 3), (4, 100, 64, -1),
                ((1 << 22) + 1, 100, 64, 0), (1 << 20, 100, 4096, 0), (4, 1 << 31, 64, 0), (4, 100, (1 << 18) + 64, 0)):
        assert size(*bad) == 0, bad


def test_head_refusals():
    L = q.lib()
    names = ("X", "M", "W", "V", "K", "t", "weight", "loss", "lse", "dX", "fp32", "ws", "bytes", "stream")
    good = dict(X=P, M=4, W=P, V=100, K=64, t=P, weight=P, loss=P, lse=P, dX=P, fp32=0, ws=P, bytes=BIG, stream=None)

    def f(**k):
        return L.qlora_head_cross_entropy(*[{**good, **k}[n] for n in names])

    for bad, want in (({"X": None}, INVALID), ({"X": ODD}, INVALID), ({"W": None}, INVALID), ({"t": None}, INVALID), ({"t": ODD}, INVALID),
                      ({"weight": ODD}, INVALID), ({"loss": None}, INVALID), ({"lse": ODD}, INVALID), ({"dX": ODD}, INVALID),
                      ({"fp32": 2}, INVALID), ({"fp32": -1}, INVALID), ({"M": -1}, INVALID), ({"V": 0}, INVALID), ({"K": 72}, SHAPE),
                      ({"M": 1 << 23}, SHAPE), ({"V": 1 << 31}, SHAPE), ({"ws": None}, WS), ({"ws": ODD}, WS), ({"bytes": 256}, WS)):
        assert f(**bad) == want, bad
    assert f(M=0, X=None, t=None, loss=None, lse=None, dX=None, ws=None, bytes=0) == OK
    assert L.qlora_head_scale(None, 4, 100, 64, P, P, P, None) == INVALID
    assert L.qlora_head_scale(P, 4, 100, 64, P, None, P, None) == INVALID
    assert L.qlora_head_scale(P, 4, 100, 64, P, P, ODD, None) == INVALID
    assert L.qlora_head_scale(P, 4, 100, 65, P, P, P, None) == SHAPE
    assert L.qlora_head_scale(None, 0, 100, 64, None, None, None, None) == OK
    names = ("X", "M", "W", "V", "K", "t", "lse", "weight", "dW", "ws", "bytes", "stream")

    def d(**k):
        return L.qlora_head_cross_entropy_dW(*[{**good, "dW": P, **k}[n] for n in names])

    for bad, want in (({"dW": None}, INVALID), ({"lse": None}, INVALID), ({"X": None}, INVALID), ({"K": 32}, SHAPE), ({"bytes": 64}, WS)):
        assert d(**bad) == want, bad
    assert d(M=0, X=None, t=None, lse=None, ws=None, bytes=0) == OK


def _tensors(*rows):
    return struct.pack("%dq" % (4 * len(rows)), *[v for r in rows for v in r])


def test_grad_norm_refusals():
    L = q.lib()
    one = _tensors((0x20000, 0x20000, 100, 1))
    size = L.qlora_grad_norm_workspace_bytes
    assert size(1, one, 1) > 0 and size(0, None, 1) == 0 and size(1, _tensors((0, 0, 0, 1)), 1) == 0
    for bad in ((-1, one, 1), (1, None, 1), (1, one, 0), (1, one, 3), (1, _tensors((0x20000, 0, -1, 1)), 1), (1, one, 5000),
                (1, _tensors((0x20000, 0, 8, 3)), 1)):
        assert size(*bad) == 0, bad

    def f(t=one, n=1, groups=1, max_norm=1.0, norm=P, ws=P, b=BIG):
        return L.qlora_clip_grad_norm(n, t, groups, max_norm, norm, ws, b, None)

    for bad, want in (({"norm": None}, INVALID), ({"norm": ODD}, INVALID), ({"max_norm": -1.0}, INVALID), ({"max_norm": float("nan")}, INVALID),
                      ({"groups": 0}, INVALID), ({"n": -1}, INVALID), ({"t": None}, INVALID), ({"groups": 3}, SHAPE), ({"n": 1 << 17}, SHAPE),
                      ({"t": _tensors((0, 0x20000, 8, 1))}, INVALID), ({"t": _tensors((0x20000, 0, 8, 1))}, INVALID),
                      ({"t": _tensors((0x20001, 0x20000, 8, 1))}, INVALID), ({"t": _tensors((0x20002, 0x20000, 8, 0))}, INVALID),
                      ({"t": _tensors((0x20000, 0x20002, 8, 0))}, INVALID), ({"ws": None}, WS), ({"ws": ODD}, WS), ({"b": 8}, WS)):
        assert f(**bad) == want, bad
    assert L.qlora_grad_norm(1, _tensors((0, 0, 8, 1)), 1, P, P, BIG, None) == INVALID
    assert L.qlora_grad_norm(1, one, 1, None, P, BIG, None) == INVALID


def test_declared_and_exported():
    for name in ("qlora_adapter_linear_workspace_bytes", "qlora_adapter_linear_fwd", "qlora_adapter_linear_bwd", "qlora_head_workspace_bytes",
                 "qlora_head_cross_entropy", "qlora_head_scale", "qlora_head_cross_entropy_dW", "qlora_grad_norm_workspace_bytes",
                 "qlora_grad_norm", "qlora_clip_grad_norm"):
        assert name in _capi.EXPORTED and getattr(q.lib(), name)
    for name in ("adapter_linear_fwd", "adapter_linear_bwd", "AdapterLinear", "AdapterLinearFn", "head_cross_entropy_fwd", "head_cross_entropy",
                 "head_cross_entropy_dW", "HeadCrossEntropyFn", "grad_norm", "clip_grad_norm"):
        assert name in q.__all__ and hasattr(q, name)
