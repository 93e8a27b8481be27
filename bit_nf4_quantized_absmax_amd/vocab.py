"""Losses over the vocabulary: log probabilities of given tokens with entropy
and alternatives, and distillation from a teacher's top logits, each with its
gradient (formulas and rules in the C ABI's header).  Argument marshalling
only, as in ops.py.

Logits are [M, V] device tensors in bfloat16, float16 or float32 whose rows
are contiguous; the row pitch is free (a padded vocabulary: logits[:, :V])."""

import ctypes
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from ._capi import LogitsStruct, TeacherStruct, check, lib
from .ops import _need, _ptr, _stream, _workspace

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor                    # float32 [M]
    entropy: torch.Tensor                    # float32 [M]
    lse: torch.Tensor                        # float32 [M, 2]: (largest logit, rest); their sum is the log-sum-exp
    top_logprob: Optional[torch.Tensor]      # float32 [M, top]
    top_index: Optional[torch.Tensor]        # int64 [M, top]


def _rows(z, name):
    """Shape and row pitch of a [M, V] device tensor with contiguous rows."""
    if not isinstance(z, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if z.device.type != "cuda":
        raise ValueError("%s must be on a GPU device" % name)
    if z.dtype not in TYPES:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, z.dtype))
    if z.dim() != 2 or z.shape[1] < 1:
        raise ValueError("%s must be 2-D [tokens, words]" % name)
    M, V = z.shape
    if V > 1 and z.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if M > 1 and z.stride(0) < V:
        raise ValueError("%s has overlapping rows" % name)
    return M, V, z.stride(0) if M > 1 else V


def _logits(z):
    M, V, pitch = _rows(z, "logits")
    return M, V, LogitsStruct(z.data_ptr(), TYPES[z.dtype], M, V, pitch)


def _grad_rows(z, out):
    """The gradient's tensor and pitch: the caller's `out` (which may be z
    itself), or a fresh one whose rows start at the same place within 16 bytes
    as z's, so that both are moved 16 bytes at a time."""
    M, V = z.shape
    if out is None:
        each = 16 // z.element_size()
        pitch = V + ((z.stride(0) - V) % each if M > 1 else 0)
        return torch.empty(M, pitch, dtype=z.dtype, device=z.device)[:, :V], pitch
    oM, oV, pitch = _rows(out, "out")
    if out.dtype != z.dtype or (oM, oV) != (M, V):
        raise ValueError("out must be %s %s" % (z.dtype, (M, V)))
    return out, pitch


def _row_values(t, name, M):
    if t is not None:
        _need(t, torch.float32, name, (M,))
    return _ptr(t)


def token_logprobs(logits, target, top=0, workspace=None):
    """Log probabilities of the words target [M] (int64; a value outside
    [0, V) has none and gives 0), the entropy and log-sum-exp of every row, and
    its `top` (at most 64) most likely words, the lower index first among equal
    logits (qlora_token_logprobs)."""
    M, V, st = _logits(logits)
    _need(target, torch.int64, "target", (M,))
    dev = logits.device
    logprob = torch.empty(M, dtype=torch.float32, device=dev)     # their own storage: a view's base keeps it from being
    entropy = torch.empty(M, dtype=torch.float32, device=dev)     # changed in place under autograd
    lse = torch.empty(M, 2, dtype=torch.float32, device=dev)
    top_logprob = top_index = None
    if top:
        if not 0 <= top <= min(64, V):
            raise ValueError("top must be at most 64 and at most the number of words")
        top_logprob = torch.empty(M, top, dtype=torch.float32, device=dev)
        top_index = torch.empty(M, top, dtype=torch.int64, device=dev)
    ws, ws_bytes = _workspace(workspace, lib().qlora_vocab_workspace_bytes(st.type, M, V, top), dev)
    check(lib().qlora_token_logprobs(ctypes.byref(st), _ptr(target), top, _ptr(logprob), _ptr(entropy), _ptr(lse),
                                     _ptr(top_logprob), _ptr(top_index), _ptr(ws), ws_bytes, _stream(logits)),
          "qlora_token_logprobs")
    return TokenLogprobs(logprob, entropy, lse, top_logprob, top_index)


def token_logprobs_bwd(logits, target, lse, entropy, g_logprob=None, g_entropy=None, out=None):
    """The gradient [M, V] of the logits, in their type, from those of the log
    probabilities and of the entropy (float32 [M], None: 0); lse and entropy as
    token_logprobs returned them.  out may be the logits themselves."""
    M, V, st = _logits(logits)
    _need(target, torch.int64, "target", (M,))
    _need(lse, torch.float32, "lse", (M, 2))
    _need(entropy, torch.float32, "entropy", (M,))
    gl, gh = _row_values(g_logprob, "g_logprob", M), _row_values(g_entropy, "g_entropy", M)
    dz, pitch = _grad_rows(logits, out)
    check(lib().qlora_token_logprobs_bwd(ctypes.byref(st), _ptr(target), _ptr(lse), _ptr(entropy), gl, gh, _ptr(dz),
                                         pitch, _stream(logits)), "qlora_token_logprobs_bwd")
    return dz


def _teacher(index, logit, temperature, M):
    if not isinstance(index, torch.Tensor) or index.dim() != 2:
        raise ValueError("index must be a tensor [tokens, entries]")
    K = index.shape[1]
    if not 1 <= K <= 256:
        raise ValueError("1 to 256 teacher entries a token")
    _need(index, torch.int64, "index", (M, K))
    _need(logit, torch.float32, "logit", (M, K))
    return TeacherStruct(index.data_ptr(), logit.data_ptr(), K, float(temperature))


def distill_topk_fwd(logits, index, logit, temperature=1.0, workspace=None):
    """KL(teacher || student) per row at a temperature, the teacher known by
    its words index [M, K] (int64; outside [0, V): no entry) and their logits
    [M, K] (float32).  Returns (loss [M], lse [M, 2], the pair of token_logprobs at
    this temperature) (qlora_distill_fwd)."""
    M, V, st = _logits(logits)
    te = _teacher(index, logit, temperature, M)
    loss = torch.empty(M, dtype=torch.float32, device=logits.device)
    lse = torch.empty(M, 2, dtype=torch.float32, device=logits.device)
    ws, ws_bytes = _workspace(workspace, lib().qlora_vocab_workspace_bytes(st.type, M, V, 0), logits.device)
    check(lib().qlora_distill_fwd(ctypes.byref(st), ctypes.byref(te), _ptr(loss), _ptr(lse), _ptr(ws), ws_bytes,
                                  _stream(logits)), "qlora_distill_fwd")
    return loss, lse


def distill_topk_bwd(logits, index, logit, temperature, lse, weight=None, out=None):
    """The gradient of the logits, in their type, for gradients weight [M]
    (float32, None: 1) of the losses (qlora_distill_bwd).  out may be the
    logits themselves."""
    M, V, st = _logits(logits)
    te = _teacher(index, logit, temperature, M)
    _need(lse, torch.float32, "lse", (M, 2))
    gw = _row_values(weight, "weight", M)
    dz, pitch = _grad_rows(logits, out)
    check(lib().qlora_distill_bwd(ctypes.byref(st), ctypes.byref(te), _ptr(lse), gw, _ptr(dz), pitch,
                                  _stream(logits)), "qlora_distill_bwd")
    return dz


def distill_topk(logits, index, logit, temperature=1.0, weight=None, out=None, workspace=None):
    """Loss and gradient in one call, for a step whose loss is the sum of
    weight * loss: returns (loss [M], dlogits [M, V]) (qlora_distill)."""
    M, V, st = _logits(logits)
    te = _teacher(index, logit, temperature, M)
    gw = _row_values(weight, "weight", M)
    dz, pitch = _grad_rows(logits, out)
    loss = torch.empty(M, dtype=torch.float32, device=logits.device)
    lse = torch.empty(M, 2, dtype=torch.float32, device=logits.device)
    ws, ws_bytes = _workspace(workspace, lib().qlora_vocab_workspace_bytes(st.type, M, V, 0), logits.device)
    check(lib().qlora_distill(ctypes.byref(st), ctypes.byref(te), gw, _ptr(loss), _ptr(lse), _ptr(dz), pitch,
                              _ptr(ws), ws_bytes, _stream(logits)), "qlora_distill")
    return loss, dz


class TokenLogprobsFn(torch.autograd.Function):
    """(logprob [M], entropy [M]) of logits [M, V] and target [M], differentiable in the logits."""

    @staticmethod
    def forward(ctx, logits, target):
        r = token_logprobs(logits, target)
        ctx.save_for_backward(logits, target, r.lse, r.entropy)
        return r.logprob, r.entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logprob, g_entropy):
        logits, target, lse, entropy = ctx.saved_tensors
        return token_logprobs_bwd(logits, target, lse, entropy, g_logprob.contiguous(), g_entropy.contiguous()), None


class DistillTopKFn(torch.autograd.Function):
    """loss [M] of logits [M, V] against a teacher's top logits, differentiable in the logits."""

    @staticmethod
    def forward(ctx, logits, index, logit, temperature):
        loss, lse = distill_topk_fwd(logits, index, logit, temperature)
        ctx.save_for_backward(logits, index, logit, lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        logits, index, logit, lse = ctx.saved_tensors
        return distill_topk_bwd(logits, index, logit, ctx.temperature, lse, g.contiguous()), None, None, None
