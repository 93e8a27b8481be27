"""The norm of many gradients and clipping by it (formulas and rules in the C
ABI's header).  Argument marshalling only, as in ops.py; a model's gradients are
hundreds of small tensors, so they are looked at attribute by attribute, over
the whole list at a time."""

import struct
from operator import attrgetter

import torch
from torch.autograd.graph import increment_version

from ._capi import check, lib
from .adapters import _on
from .ops import _ptr, _stream, _workspace

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
PLAIN = {torch.Tensor, torch.nn.Parameter}

_dtype = attrgetter("dtype")


def _listed(tensors, name):
    """(data pointers, element counts, types, device index or None) of a list of tensors."""
    if not set(map(type, tensors)) <= PLAIN and not all(isinstance(t, torch.Tensor) for t in tensors):
        raise TypeError("%s must be tensors" % name)
    types = list(map(_dtype, tensors))
    for t in set(types) - TYPES.keys():
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t))
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        raise ValueError("%s must be contiguous" % name)
    devices = set(map(torch.Tensor.get_device, tensors))
    if len(devices) > 1 or -1 in devices:
        raise ValueError("%s must be on one GPU device" % name)
    return (list(map(torch.Tensor.data_ptr, tensors)), list(map(torch.Tensor.numel, tensors)), list(map(TYPES.get, types)),
            devices.pop() if devices else None)


def _call(grads, max_norm, groups, out, workspace):
    grads = list(grads)
    ptrs, counts, types, device = _listed(grads, "grads")
    groups = int(groups)
    if groups < 1:
        raise ValueError("groups must be at least 1")
    if device is None:
        raise ValueError("no gradients: the norm has no device to go to")
    if groups > 1:
        for t in grads:
            if t.dim() == 0 or t.shape[0] % groups:
                raise ValueError("every gradient's first axis must hold %d equal parts, got shape %s" % (groups, tuple(t.shape)))
    to = ptrs
    if max_norm is not None:
        written = grads if out is None else list(out)
        if out is not None:
            to, to_counts, to_types, to_device = _listed(written, "out")
            if to_types != types or to_counts != counts or to_device != device:
                raise ValueError("out must be one tensor of the same size, type and device for every gradient")
        if len(set(to)) != len(to):
            used = [p for p, n in zip(to, counts) if n]
            if len(set(used)) != len(used):
                raise ValueError("a tensor is written twice")
    n = len(grads)
    flat = [0] * (4 * n)
    flat[0::4], flat[1::4], flat[2::4], flat[3::4] = ptrs, to, counts, types
    table = struct.pack("%dq" % (4 * n), *flat)     # qlora_grad_tensor [n]
    first = grads[0]
    norm = torch.empty(groups, dtype=torch.float32, device=first.device)
    ws, ws_bytes = _workspace(workspace, lib().qlora_grad_norm_workspace_bytes(n, table, groups), first.device)
    with _on(first.device, ws):
        if max_norm is None:
            check(lib().qlora_grad_norm(n, table, groups, _ptr(norm), _ptr(ws), ws_bytes, _stream(first)), "qlora_grad_norm")
        else:
            check(lib().qlora_clip_grad_norm(n, table, groups, float(max_norm), _ptr(norm), _ptr(ws), ws_bytes, _stream(first)),
                  "qlora_clip_grad_norm")
            increment_version(written)   # to autograd a change like that of torch's own in-place calls
    return norm


def grad_norm(grads, groups=1, workspace=None):
    """The norm (float32 [groups]) of the elements of all tensors (float32,
    bfloat16 or float16, contiguous, on one device).  groups > 1: every tensor's
    first axis holds that many equal parts, as stacked adapters' gradients do, and
    part g counts for norm g (qlora_grad_norm)."""
    return _call(grads, None, groups, None, workspace)


def clip_grad_norm(grads, max_norm, groups=1, out=None, workspace=None):
    """grad_norm, and the gradients times min(1, max_norm / (norm + 1e-6)), in
    place or into `out` (for every gradient a tensor of its size and type, which
    overlaps no gradient but its own).  Returns the norms before clipping (qlora_clip_grad_norm)."""
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError("max_norm must not be negative or NaN")
    return _call(grads, max_norm, groups, out, workspace)
