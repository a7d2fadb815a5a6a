"""Layer norm over the rows of a matrix and its gradients (include/layer_norm.h)."""
from __future__ import annotations

import ctypes
import struct

import torch

from . import LN_EXPORTED, SgemmError, _on_stream, lib
from .f8 import _TYPE, _rows, _stream_here

__all__ = ["layer_norm", "layer_norm_backward", "layer_norm_backward_workspace_size", "LN_EXPORTED"]

# layer_norm_args and layer_norm_backward_args
_forward_args = struct.Struct("@iiPiiPPifPiPPP").pack
_backward_args = struct.Struct("@iiPiPiiPPPiPiPPfP").pack


def _vector(name, t, n, at):
    """The address and type of a vector of n parameters on device `at`."""
    kind = _TYPE.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    if t.get_device() != at:
        raise ValueError(f"{name} is on another device")
    return t.data_ptr(), kind


def _numbers(name, t, n, at):
    """The address of n FP32 numbers on device `at`."""
    address, kind = _vector(name, t, n, at)
    if kind != 0:
        raise TypeError(f"{name} must be float32")
    return address


def _like(name, t, x):
    """The row stride of a matrix of x's shape and type."""
    if t.dtype is not x.dtype:
        raise TypeError(f"{name} has another type than x")
    if t.shape != x.shape:
        raise ValueError("shape mismatch")
    if t.get_device() != x.get_device():
        raise ValueError(f"{name} is on another device")
    return _rows(name, t)[2]


def _matrix(x):
    """(type, rows, columns, row stride, device index, stream) of x."""
    kind = _TYPE.get(x.dtype)
    if kind is None:
        raise TypeError("x must be float32, bfloat16 or float16")
    rows, cols, ld = _rows("x", x)
    if cols < 1:
        raise ValueError("rows must have elements")
    return kind, rows, cols, ld, *_stream_here("x", x)


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, stats=False, out=None, stream=None):
    """(x - mean) * rstd * weight + bias along the rows of a 2-D CUDA tensor (float32, bfloat16,
    float16), rounded once to x's type, with rstd = 1 / sqrt(variance + eps). weight and bias: vectors
    of one type, 1 and 0 if left out. With stats returns (y, mean, rstd), mean and rstd in float32, for
    layer_norm_backward. out: where to write y (x itself for in place). `stream`: where to run (a torch
    stream or a handle; the current stream unless given), new results belong to it. Raises SgemmError
    on a nonzero status."""
    if stream is not None:
        return _on_stream(stream, lambda: layer_norm(x, weight, bias, eps=eps, stats=stats, out=out),
                          [t for t in (x, weight, bias, out) if t is not None])
    kind, rows, cols, ldx, at, handle = _matrix(x)
    wp = bp = wt = mp = rp = 0
    if weight is not None:
        wp, wt = _vector("weight", weight, cols, at)
    if bias is not None:
        bp, bt = _vector("bias", bias, cols, at)
        if weight is not None and wt != bt:
            raise TypeError("weight and bias must have one type")
        wt = bt
    if out is None:
        out = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
        ldy = cols
    else:
        ldy = _like("out", out, x)
    if stats:
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    rc = lib.layer_norm_with(_forward_args(rows, cols, x.data_ptr(), kind, ldx, wp, bp, wt, eps,
                                           out.data_ptr(), ldy, mp, rp, handle))
    if rc != 0:
        raise SgemmError(rc, "layer_norm")
    return (out, mean, rstd) if stats else out


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, out=None, dweight=None, dbias=None,
                        beta=0.0, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm from dy, that of its result: dx in x's type, those
    of the weight and the bias in float32, summed over the rows and added to beta times what dweight
    and dbias hold if these are given. out: where to write dx (dy or x itself for in place). Without a
    weight (all ones) and without dweight and dbias, these two are None. `stream` as in layer_norm."""
    if stream is not None:
        return _on_stream(stream, lambda: layer_norm_backward(
            dy, x, mean, rstd, weight, out=out, dweight=dweight, dbias=dbias, beta=beta),
            [t for t in (dy, x, mean, rstd, weight, out, dweight, dbias) if t is not None])
    kind, rows, cols, ldx, at, handle = _matrix(x)
    lddy = _like("dy", dy, x)
    if mean is None or rstd is None:
        raise TypeError("mean and rstd are needed")
    mp, rp = _numbers("mean", mean, rows, at), _numbers("rstd", rstd, rows, at)
    if beta != 0.0 and (dweight is None or dbias is None):
        raise ValueError("beta needs dweight and dbias to scale")
    wp = wt = dwp = dbp = 0
    if weight is not None:
        wp, wt = _vector("weight", weight, cols, at)
    if weight is not None or dweight is not None or dbias is not None:
        if dweight is None:
            dweight = torch.empty(cols, dtype=torch.float32, device=x.device)
        if dbias is None:
            dbias = torch.empty(cols, dtype=torch.float32, device=x.device)
        dwp, dbp = _numbers("dweight", dweight, cols, at), _numbers("dbias", dbias, cols, at)
        if -4 * cols < dwp - dbp < 4 * cols:
            raise ValueError("dweight and dbias overlap")
    if out is None:
        out = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
        lddx = cols
    else:
        lddx = _like("out", out, x)
    rc = lib.layer_norm_backward_with(_backward_args(
        rows, cols, dy.data_ptr(), lddy, x.data_ptr(), kind, ldx, mp, rp, wp, wt, out.data_ptr(), lddx,
        dwp, dbp, beta, handle))
    if rc != 0:
        raise SgemmError(rc, "layer_norm_backward")
    return out, dweight, dbias


def layer_norm_backward_workspace_size(rows, cols) -> tuple[int, int]:
    """(status, bytes)."""
    n = ctypes.c_size_t(0)
    rc = lib.layer_norm_backward_workspace_size(rows, cols, ctypes.byref(n))
    return rc, n.value
