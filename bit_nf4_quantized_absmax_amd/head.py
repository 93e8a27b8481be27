"""Softmax cross entropy through a frozen output head without the logits, with
the gradients of the hidden states and, where it is tuned as well, of the head
(formulas and rules in the C ABI's header).  Argument marshalling only, as in
ops.py."""

import torch
from torch.autograd.function import once_differentiable

from ._capi import check, lib
from .adapters import _on, _written
from .ops import _mat, _need, _out, _ptr, _stream, _workspace

LOSS, DX, DW = 0, 1, 2   # qlora_head_pass


def _checks(X, W, target, weight):
    M, K = _mat(X, "X")
    V = _mat(W, "W")[0]
    if W.shape[1] != K:
        raise ValueError("W must be [V, %d]" % K)
    _need(target, torch.int64, "target", (M,))
    if weight is not None:
        _need(weight, torch.float32, "weight", (M,))
    return M, V, K


def _forward(X, W, target, weight, dX, workspace):
    M, V, K = _checks(X, W, target, weight)
    dev = X.device
    loss = torch.empty(M, dtype=torch.float32, device=dev)
    lse = torch.empty(M, 2, dtype=torch.float32, device=dev)
    need = lib().qlora_head_workspace_bytes(M, V, K, LOSS if dX is None else DX)
    ws, ws_bytes = _workspace(workspace, need, dev)
    with _on(dev, W, target, weight, dX, ws):
        check(lib().qlora_head_cross_entropy(_ptr(X), M, _ptr(W), V, K, _ptr(target), _ptr(weight), _ptr(loss), _ptr(lse), _ptr(dX),
                                             int(dX is not None and dX.dtype == torch.float32), _ptr(ws), ws_bytes, _stream(X)),
              "qlora_head_cross_entropy")
    return loss, lse


def head_cross_entropy_fwd(X, W, target, workspace=None):
    """Losses log sum_j e^z_mj - z_m,target, z = X W^T, of hidden states X [M, K]
    and a head W [V, K] in bf16; target int64 [M] (outside [0, V): loss 0).
    Returns (loss [M], lse [M, 2]), the sum of lse's pair being the log-sum-exp;
    head_cross_entropy_dW takes the pairs as they are (qlora_head_cross_entropy)."""
    return _forward(X, W, target, None, None, workspace)


def head_cross_entropy(X, W, target, weight=None, dX_out=None, workspace=None):
    """Loss and gradient in one call, for a step whose loss is the sum of weight *
    loss (weight float32 [M], None: 1): returns (loss [M], lse [M, 2], dX [M, K]).
    dX_out may be bfloat16 (the default) or float32 (qlora_head_cross_entropy)."""
    dtype = dX_out.dtype if isinstance(dX_out, torch.Tensor) and dX_out.dtype == torch.float32 else torch.bfloat16
    M, K = _mat(X, "X")
    dX = _out(dX_out, (M, K), X.device, "dX", dtype)
    loss, lse = _forward(X, W, target, weight, dX, workspace)
    _written(dX_out)
    return loss, lse, dX


def head_cross_entropy_dW(X, W, target, lse, weight=None, dW_out=None, workspace=None):
    """The gradient [V, K] of the head for gradients weight [M] of the losses, from
    the lse that either call above returned (qlora_head_cross_entropy_dW)."""
    M, V, K = _checks(X, W, target, weight)
    _need(lse, torch.float32, "lse", (M, 2))
    dev = X.device
    dW = _out(dW_out, (V, K), dev, "dW")
    ws, ws_bytes = _workspace(workspace, lib().qlora_head_workspace_bytes(M, V, K, DW), dev)
    with _on(dev, W, target, lse, weight, dW, ws):
        check(lib().qlora_head_cross_entropy_dW(_ptr(X), M, _ptr(W), V, K, _ptr(target), _ptr(lse), _ptr(weight), _ptr(dW), _ptr(ws),
                                                ws_bytes, _stream(X)), "qlora_head_cross_entropy_dW")
    if M == 0:   # the call above writes nothing then
        dW.zero_()
    _written(dW_out)
    return dW


class HeadCrossEntropyFn(torch.autograd.Function):
    """loss [M] of hidden states X, differentiable in X and, where it asks for a
    gradient, in W.  The forward pass makes X's gradient at weight 1 along with
    the losses and keeps it in float32; the backward pass scales it."""

    @staticmethod
    def forward(ctx, X, W, target):
        D = None
        if ctx.needs_input_grad[0]:
            D = torch.empty(X.shape, dtype=torch.float32, device=X.device)
            loss, lse, _ = head_cross_entropy(X, W, target, dX_out=D)
        else:
            loss, lse = head_cross_entropy_fwd(X, W, target)
        if ctx.needs_input_grad[1]:
            ctx.save_for_backward(X, W, target, lse, D)
        else:
            ctx.save_for_backward(None, W, target, None, D)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        X, W, target, lse, D = ctx.saved_tensors
        g = g.contiguous()
        dX = dW = None
        if ctx.needs_input_grad[0]:
            M, K = D.shape
            dX = torch.empty(M, K, dtype=torch.bfloat16, device=D.device)
            with _on(D.device, g):
                check(lib().qlora_head_scale(_ptr(D), M, W.shape[0], K, _ptr(target), _ptr(g), _ptr(dX), _stream(D)), "qlora_head_scale")
        if ctx.needs_input_grad[1]:
            dW = head_cross_entropy_dW(X, W, target, lse, weight=g)
        return dX, dW, None
