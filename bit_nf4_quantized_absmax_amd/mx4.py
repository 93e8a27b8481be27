"""MX4 arrays (blocks of 32 E2M1 codes under a power-of-two scale) and the
linear layer on an MX4 weight; the C ABI's header states the format and the
rules.  Argument marshalling only, as in ops.py."""

import ctypes
from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from ._capi import MX4ArrayStruct, check, lib
from .ops import _mat, _need, _out, _ptr, _stream, _workspace

IN_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


@dataclass
class MX4Tensor:
    """An array [rows, cols] in MX4 (cols % 32 == 0; Kp: cols filled up to a multiple of 256).

    codes uint8 [rows, Kp / 2], scales uint8 [Kp / 256, rows, 8]: the bytes of
    the 8 blocks of a 256-wide slab of a row (qlora_mx4_array).
    """
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def device(self):
        return self.codes.device

    def struct(self):
        slabs = (self.cols + 255) // 256
        _need(self.codes, torch.uint8, "codes", (self.rows, 128 * slabs))
        _need(self.scales, torch.uint8, "scales", (slabs, self.rows, 8))
        return self._unchecked()

    def _unchecked(self):
        return MX4ArrayStruct(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols)

    @classmethod
    def empty(cls, rows, cols, device):
        slabs = (cols + 255) // 256
        return cls(torch.empty(rows, 128 * slabs, dtype=torch.uint8, device=device),
                   torch.empty(slabs, rows, 8, dtype=torch.uint8, device=device), rows, cols)

    @classmethod
    def quantize(cls, X, out=None):
        """A float32, bfloat16 or float16 device tensor [rows, cols] in MX4
        (qlora_mx4_quantize), into `out` when given."""
        in_type = IN_TYPES.get(X.dtype)
        if in_type is None:
            raise TypeError("X must be float32, bfloat16 or float16, got %s" % X.dtype)
        rows, cols = _mat(X, "X", X.dtype)
        if out is None:
            out = cls.empty(rows, cols, X.device)
            st = out._unchecked()
        else:
            if out.shape != (rows, cols):
                raise ValueError("out has shape %s, expected %s" % (out.shape, (rows, cols)))
            st = out.struct()
        check(lib().qlora_mx4_quantize(_ptr(X), in_type, ctypes.byref(st), _stream(X)), "qlora_mx4_quantize")
        return out

    def dequantize(self, out=None):
        """The values as bf16 [rows, cols], exact (qlora_mx4_dequantize)."""
        out = _out(out, (self.rows, self.cols), self.device, "out")
        st = self.struct()
        check(lib().qlora_mx4_dequantize(ctypes.byref(st), _ptr(out), _stream(out)), "qlora_mx4_dequantize")
        return out

    def nbytes(self):
        return self.codes.numel() + self.scales.numel()


def mx4_matmul(X, w, T=None, B=None, out=None):
    """Y = X W^T (+ T B^T) of two MX4Tensors X [M, K] and w [N, K], with T
    [M, r] and B [N, r] in bf16 (qlora_mx4_matmul)."""
    r = 0
    if (T is None) != (B is None):
        raise ValueError("T and B come together")
    if B is not None:
        r = _mat(B, "B")[1]
        _need(B, torch.bfloat16, "B", (w.rows, r))
        _need(T, torch.bfloat16, "T", (X.rows, r))
    Y = _out(out, (X.rows, w.rows), X.device, "Y")
    xs, ws = X.struct(), w.struct()
    check(lib().qlora_mx4_matmul(ctypes.byref(xs), ctypes.byref(ws), _ptr(T), _ptr(B), r, _ptr(Y), _stream(Y)),
          "qlora_mx4_matmul")
    return Y


def _checks(X, w, A, B):
    M, K = _mat(X, "X")
    if K != w.cols:
        raise ValueError("X must be [M, %d]" % w.cols)
    if A is None and B is None:
        return M, w.rows, K, 0
    if A is None or B is None:
        raise ValueError("A and B come together")
    r = _mat(A, "A")[0]
    _need(A, torch.bfloat16, "A", (r, K))
    _need(B, torch.bfloat16, "B", (w.rows, r))
    return M, w.rows, K, r


def mx4_linear_fwd(X, w, A=None, B=None, scale=1.0, T_out=None, out=None, workspace=None):
    """Y = Q(X) W^T + scale (X A^T) B^T with W an MX4Tensor and X bf16, rounded
    to MX4 for the frozen product; returns (Y, T), T = scale X A^T [M, r] (None
    without a LoRA pair)."""
    M, N, K, r = _checks(X, w, A, B)
    Y = _out(out, (M, N), X.device, "Y")
    T = _out(T_out, (M, r), X.device, "T") if r else None
    ws, ws_bytes = _workspace(workspace, lib().qlora_mx4_linear_workspace_bytes(M, N, K, r, 0), X.device)
    st = w.struct()
    check(lib().qlora_mx4_linear_fwd(_ptr(X), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(scale), _ptr(Y),
                                     _ptr(T), _ptr(ws), ws_bytes, _stream(X)), "qlora_mx4_linear_fwd")
    return Y, T


def mx4_linear_bwd(dY, X, T, w, A, B, scale, need_dX=True, need_dA=True, need_dB=True, workspace=None,
                   dX_out=None, dA_out=None, dB_out=None):
    """(dX, dA, dB) of mx4_linear_fwd with a LoRA pair (None where not
    requested); T as returned by it, or None (recomputed).  The rounding of X
    passes its gradient straight through.  Without tokens dA and dB are zero,
    also where the caller gave their storage."""
    if A is None or B is None:
        raise ValueError("the backward pass needs a LoRA pair")
    M, N, K, r = _checks(X, w, A, B)
    _need(dY, torch.bfloat16, "dY", (M, N))
    if T is not None:
        _need(T, torch.bfloat16, "T", (M, r))
    dev = X.device
    dX = _out(dX_out, (M, K), dev, "dX") if need_dX else None
    dA = _out(dA_out, (r, K), dev, "dA") if need_dA else None
    dB = _out(dB_out, (N, r), dev, "dB") if need_dB else None
    ws, ws_bytes = _workspace(workspace, lib().qlora_mx4_linear_workspace_bytes(M, N, K, r, 1), dev)
    st = w.struct()
    check(lib().qlora_mx4_linear_bwd(_ptr(dY), _ptr(X), _ptr(T), M, ctypes.byref(st), _ptr(A), _ptr(B), r,
                                     float(scale), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws_bytes, _stream(X)),
          "qlora_mx4_linear_bwd")
    if M == 0:   # the call above writes nothing then
        for d in (dA, dB):
            if d is not None:
                d.zero_()
    return dX, dA, dB


class MX4LinearFn(torch.autograd.Function):
    """mx4_linear_fwd with gradients for X, A and B only."""

    @staticmethod
    def forward(ctx, X, A, B, w, scale):
        Y, T = mx4_linear_fwd(X, w, A, B, scale)
        ctx.save_for_backward(X, A, B, T)
        ctx.w, ctx.scale = w, scale
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, A, B, T = ctx.saved_tensors
        dX, dA, dB = mx4_linear_bwd(dY.contiguous(), X, T, ctx.w, A, B, ctx.scale,
                                    need_dX=ctx.needs_input_grad[0], need_dA=ctx.needs_input_grad[1],
                                    need_dB=ctx.needs_input_grad[2])
        return dX, dA, dB, None, None


class MX4Linear(torch.nn.Module):
    """QLoRALinear on an MX4 weight: a frozen MX4 base, activations rounded to
    MX4 for it, and a trainable LoRA pair in bf16."""

    def __init__(self, weight, r, alpha, lora_A=None, lora_B=None):
        super().__init__()
        self.w = MX4Tensor.quantize(weight.contiguous())
        N, K = self.w.shape
        dev = weight.device
        self.r = int(r)
        self.scale = float(torch.tensor(alpha, dtype=torch.float32) / torch.tensor(r, dtype=torch.float32))
        self.lora_A = torch.nn.Parameter(lora_A if lora_A is not None else
                                         torch.zeros(r, K, dtype=torch.bfloat16, device=dev))
        self.lora_B = torch.nn.Parameter(lora_B if lora_B is not None else
                                         torch.zeros(N, r, dtype=torch.bfloat16, device=dev))

    def forward(self, x):
        lead = x.shape[:-1]
        y = MX4LinearFn.apply(x.reshape(-1, x.shape[-1]).contiguous(), self.lora_A, self.lora_B, self.w, self.scale)
        return y.reshape(*lead, y.shape[-1])
