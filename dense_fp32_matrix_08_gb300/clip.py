"""The norm of all gradients together, and clipping by it (include/grad_clip.h)."""
from __future__ import annotations

from array import array
from operator import attrgetter

import torch

from . import GC_EXPORTED, SgemmError, _on_stream, _stream, lib
from .f8 import _TYPE

__all__ = ["clip_grad_norm", "GC_EXPORTED"]


_dtype = attrgetter("dtype")
_get_device, _is_contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous


def _lists(name, tensors):
    """(addresses, types, sizes) of contiguous tensors on the current device, as arrays. (There may be
    hundreds of them: one pass of a built-in per question.)"""
    where = set(map(_get_device, tensors))  # (a TypeError for what is no tensor)
    try:
        types = array("i", map(_TYPE.__getitem__, map(_dtype, tensors)))
    except KeyError:
        raise TypeError(f"{name} must be float32, bfloat16 or float16") from None
    if -1 in where:
        raise TypeError(f"{name} must live on a CUDA device")
    if where and where != {torch.cuda.current_device()}:
        raise ValueError(f"{name} must be on the current device")
    if not all(map(_is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    return (array("Q", map(torch.Tensor.data_ptr, tensors)), types,
            array("q", map(torch.Tensor.numel, tensors)))


def clip_grad_norm(grads, max_norm, *, eps=1e-6, out=None, stream=None):
    """Scales gradients by min(1, max_norm / (norm + eps)), norm = sqrt(the sum of squares of all their
    elements), and returns that norm, a float32 tensor of no dimensions on the device. grads: contiguous
    CUDA tensors of float32, bfloat16 or float16, in any mixture. They are changed in place; with out, a
    list of as many tensors with as many elements each, those are written instead, each in its own type. With
    max_norm = inf and no out nothing is changed: only the norm is computed. `stream`: where to run (a
    torch stream or a handle; the current stream unless given), the norm belongs to it. Raises
    SgemmError on a nonzero status (-7: results that overlap, such as one gradient given twice)."""
    grads = list(grads)
    if out is not None:
        out = list(out)
    if stream is not None:
        return _on_stream(stream, lambda: clip_grad_norm(grads, max_norm, eps=eps, out=out),
                          grads + (out or []))
    at, types, sizes = _lists("grads", grads)
    to, to_types = at, types
    if out is not None:
        to, to_types, have = _lists("out", out)
        if have != sizes:
            raise ValueError("out must have as many elements as grads, tensor by tensor")
    scale = out is not None or max_norm != float("inf")
    norm = torch.empty((), dtype=torch.float32, device="cuda")
    rc = lib.clip_grad_norm(
        len(grads), at.buffer_info()[0], types.buffer_info()[0], sizes.buffer_info()[0], max_norm, eps,
        to.buffer_info()[0] if scale else None, to_types.buffer_info()[0], norm.data_ptr(), _stream(None))
    if rc != 0:
        raise SgemmError(rc, "clip_grad_norm")
    return norm
