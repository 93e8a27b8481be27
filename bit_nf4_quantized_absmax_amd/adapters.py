"""The linear layer with many LoRA adapters beside one frozen NF4 weight: every
token names the adapter of its request (formulas and rules in the C ABI's
header).  Argument marshalling only, as in ops.py."""

import contextlib
import ctypes

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from ._capi import AdaptersStruct, check, lib
from .ops import NF4Weight, _mat, _need, _out, _ptr, _stream, _workspace

_SAME_DEVICE = contextlib.nullcontext()

# The current device without torch.cuda's look at its own state first (0.1 us a
# call instead of 0.6); not part of the documented interface, as ops._raw_stream.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(device, *tensors):
    """The context in which work on `device` is launched; every tensor given (or None) has to be there."""
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors on different devices: %s and %s" % (device, t.device))
    return _SAME_DEVICE if _current_device() == index else torch.cuda.device(device)


def _written(*tensors):
    """The caller's tensors (or None) have new values: autograd learns it as from torch's own in-place
    calls, and what it had saved of them raises in backward() instead of being used."""
    given = [t for t in tensors if t is not None]
    if given:
        increment_version(given)


def _checks(X, w, A, B, scale, index):
    M, K = _mat(X, "X")
    if K != w.cols:
        raise ValueError("X must be [M, %d]" % w.cols)
    if not isinstance(A, torch.Tensor) or A.dim() != 3:
        raise ValueError("A must be a tensor [adapters, r, %d]" % K)
    n, r = A.shape[0], A.shape[1]
    _need(A, torch.bfloat16, "A", (n, r, K))
    _need(B, torch.bfloat16, "B", (n, w.rows, r))
    _need(scale, torch.float32, "scale", (n,))
    _need(index, torch.int64, "index", (M,))
    return M, w.rows, K, n, r, AdaptersStruct(A.data_ptr(), B.data_ptr(), scale.data_ptr(), index.data_ptr(), n, r)


def adapter_linear_fwd(X, w, A, B, scale, index, T_out=None, out=None, workspace=None):
    """Y_m = X_m deq(W)^T + T_m B_a^T, T_m = scale_a X_m A_a^T with a = index[m]
    (int64; outside [0, n): no adapter), w an NF4Weight, A [n, r, K] and B [n,
    N, r] in bf16, scale [n] float32.  r is a multiple of 8, at most 128 (smaller
    adapters are filled up with zeros), n at most 1023.  Returns (Y, T)
    (qlora_adapter_linear_fwd)."""
    M, N, K, n, r, st = _checks(X, w, A, B, scale, index)
    dev = X.device
    Y = _out(out, (M, N), dev, "Y")
    T = _out(T_out, (M, r), dev, "T")
    ws, ws_bytes = _workspace(workspace, lib().qlora_adapter_linear_workspace_bytes(M, N, K, n, r, 0), dev)
    wt = w.struct()
    with _on(dev, w.packed, A, B, scale, index, Y, T, ws):
        check(lib().qlora_adapter_linear_fwd(_ptr(X), M, ctypes.byref(wt), ctypes.byref(st), _ptr(Y), _ptr(T), _ptr(ws), ws_bytes,
                                             _stream(X)), "qlora_adapter_linear_fwd")
    _written(out, T_out)
    return Y, T


def adapter_linear_bwd(dY, X, T, w, A, B, scale, index, need_dX=True, need_dA=True, need_dB=True, workspace=None,
                       dX_out=None, dA_out=None, dB_out=None):
    """(dX [M, K], dA [n, r, K], dB [n, N, r]) of adapter_linear_fwd (None where
    not requested); T as returned by it, or None (recomputed).  Adapters without
    tokens have zero gradients (qlora_adapter_linear_bwd)."""
    M, N, K, n, r, st = _checks(X, w, A, B, scale, index)
    _need(dY, torch.bfloat16, "dY", (M, N))
    if T is not None:
        _need(T, torch.bfloat16, "T", (M, r))
    dev = X.device
    dX = _out(dX_out, (M, K), dev, "dX") if need_dX else None
    dA = _out(dA_out, (n, r, K), dev, "dA") if need_dA else None
    dB = _out(dB_out, (n, N, r), dev, "dB") if need_dB else None
    ws, ws_bytes = _workspace(workspace, lib().qlora_adapter_linear_workspace_bytes(M, N, K, n, r, 1), dev)
    wt = w.struct()
    with _on(dev, dY, T, w.packed, A, B, scale, index, dX, dA, dB, ws):
        check(lib().qlora_adapter_linear_bwd(_ptr(dY), _ptr(X), _ptr(T), M, ctypes.byref(wt), ctypes.byref(st), _ptr(dX), _ptr(dA),
                                             _ptr(dB), _ptr(ws), ws_bytes, _stream(X)), "qlora_adapter_linear_bwd")
    if M == 0:   # the call above writes nothing then
        for d in (dA, dB):
            if d is not None:
                d.zero_()
    _written(dX_out if need_dX else None, dA_out if need_dA else None, dB_out if need_dB else None)
    return dX, dA, dB


class AdapterLinearFn(torch.autograd.Function):
    """adapter_linear_fwd with gradients for X, A and B only."""

    @staticmethod
    def forward(ctx, X, A, B, w, scale, index):
        Y, T = adapter_linear_fwd(X, w, A, B, scale, index)
        ctx.save_for_backward(X, A, B, T, scale, index)
        ctx.w = w
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, A, B, T, scale, index = ctx.saved_tensors
        need = ctx.needs_input_grad
        dX, dA, dB = adapter_linear_bwd(dY.contiguous(), X, T, ctx.w, A, B, scale, index, need_dX=need[0], need_dA=need[1],
                                        need_dB=need[2])
        return dX, dA, dB, None, None, None


class AdapterLinear(torch.nn.Module):
    """QLoRALinear with `adapters` LoRA pairs over one frozen NF4 weight; the
    adapter of every token comes with the call.  alpha: one value, or one an adapter.
    Where they are not given, lora_B is zero and lora_A uniform within K^-1/2: with both
    at zero, so would be their gradients, for ever."""

    def __init__(self, weight, adapters, r, alpha, lora_A=None, lora_B=None):
        super().__init__()
        self.w = weight if isinstance(weight, NF4Weight) else NF4Weight.quantize(weight.contiguous())
        N, K = self.w.shape
        dev = self.w.device
        self.r = int(r)
        scale = torch.as_tensor(alpha, dtype=torch.float32, device=dev) / float(r)
        self.register_buffer("scale", scale.expand(adapters).contiguous())
        if lora_A is None:
            lora_A = torch.empty(adapters, r, K, dtype=torch.bfloat16, device=dev).uniform_(-K ** -0.5, K ** -0.5)
        self.lora_A = torch.nn.Parameter(lora_A)
        self.lora_B = torch.nn.Parameter(lora_B if lora_B is not None else
                                         torch.zeros(adapters, N, r, dtype=torch.bfloat16, device=dev))

    def _apply(self, fn, recurse=True):
        """Moves and casts as any module's, but the scales stay the float32 values that the kernels take."""
        scale = self.scale
        super()._apply(fn, recurse)
        if self.scale.dtype != torch.float32:
            self.scale = scale.to(self.scale.device)
        return self

    def forward(self, x, index):
        """x [..., K]; index int64 [...], the adapter of every token."""
        lead = x.shape[:-1]
        y = AdapterLinearFn.apply(x.reshape(-1, x.shape[-1]).contiguous(), self.lora_A, self.lora_B, self.w, self.scale,
                                  index.reshape(-1).contiguous())
        return y.reshape(*lead, y.shape[-1])
