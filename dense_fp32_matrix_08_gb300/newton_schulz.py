"""Orthogonalising updates by Newton-Schulz products (include/orthogonalize.h)."""
from __future__ import annotations

import ctypes

import torch

from . import NS_EXPORTED, SgemmError, _on_stream, _stream, lib

__all__ = ["orthogonalize", "ns_orthogonalize_workspace_size", "ns_orthogonalize_plan",
           "ns_orthogonalize_status", "NS_EXPORTED"]

_MOST = 0x7fffffff  # sizes are 32-bit
_TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _matrices(name, t):
    """(type, row stride, matrix stride) of a 2-D or 3-D CUDA tensor with unit column stride and rows
    that do not overlap."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be 2-D or 3-D")
    if t.dtype not in _TYPE:
        raise TypeError(f"{name} must be float32, bfloat16 or float16")
    if not t.is_cuda:
        raise TypeError(f"{name} must live on a CUDA device")
    rows, cols = t.shape[-2:]
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = t.stride(-2) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap (an expanded tensor or a sliding window)")
    if rows > _MOST or ld > _MOST or t.shape[0] > _MOST:
        raise ValueError(f"{name}'s sizes and row stride must be below 2^31")
    ld = ld or 1
    return _TYPE[t.dtype], ld, t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else rows * ld


def orthogonalize(g, *, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, alpha=1.0,
                  beta=0.0, out=None, out_dtype=None, stream=None):
    """out = alpha * X + beta * out, X the result of `steps` Newton-Schulz steps
    X <- a X + (b S + c S^2) X, S = X X^T, from X = g / (|g|_F + eps); coefficients = (a, b, c).
    g is a matrix or a batch of them (float32, bfloat16, float16). Without `out` a new tensor of
    out_dtype (g's type unless given) is returned. With out = the weight, alpha = -rate and
    beta = 1 - rate * decay it is the whole update. `stream`: where to run (a torch stream or a handle;
    the current stream unless given), a new result belongs to it. Raises SgemmError on a nonzero
    status."""
    if stream is not None:
        return _on_stream(stream, lambda: orthogonalize(
            g, steps=steps, coefficients=coefficients, eps=eps, alpha=alpha, beta=beta, out=out,
            out_dtype=out_dtype), (g,) if out is None else (g, out))
    gt, ldg, gs = _matrices("g", g)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs an out to scale")
        out = torch.empty(g.shape, dtype=out_dtype or g.dtype, device=g.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out has another type than out_dtype")
    ot, ldo, os_ = _matrices("out", out)
    if out.shape != g.shape:
        raise ValueError("shape mismatch")
    if out.device != g.device:
        raise ValueError("out is on another device")
    batch = g.shape[0] if g.dim() == 3 else 1
    rows, cols = g.shape[-2:]
    a, b, c = coefficients
    steps = max(-1, min(steps, 65))  # (32 bits of a larger number would be another one)
    rc = lib.ns_orthogonalize(batch, rows, cols, g.data_ptr() or None, gt, ldg, gs, steps,
                              (ctypes.c_float * 3)(a, b, c), eps, alpha, beta, out.data_ptr() or None, ot, ldo,
                              os_, _stream(None))
    if rc != 0:
        raise SgemmError(rc, "ns_orthogonalize")
    return out


def ns_orthogonalize_workspace_size(batch, rows, cols) -> tuple[int, int]:
    """(status, bytes)."""
    n = ctypes.c_size_t(0)
    rc = lib.ns_orthogonalize_workspace_size(batch, rows, cols, ctypes.byref(n))
    return rc, n.value


def ns_orthogonalize_plan(batch, rows, cols, num_sms=0) -> dict:
    """How orthogonalize runs a problem: {"tile_cols", "tiles", "whole", "split"}, the last three for
    each product of a step (see the header)."""
    cols_of, three = ctypes.c_int(0), [(ctypes.c_int * 3)() for _ in range(3)]
    rc = lib.ns_orthogonalize_plan(batch, rows, cols, num_sms, ctypes.byref(cols_of), *three)
    if rc != 0:
        raise SgemmError(rc, "ns_orthogonalize_plan")
    return {"tile_cols": cols_of.value, "tiles": tuple(three[0]), "whole": tuple(three[1]),
            "split": tuple(three[2])}


def ns_orthogonalize_status() -> tuple[int, int]:
    """(call status, device status word of ns_orthogonalize); reading clears the word."""
    v = ctypes.c_int(0)
    rc = lib.ns_orthogonalize_status(ctypes.byref(v))
    return rc, v.value
