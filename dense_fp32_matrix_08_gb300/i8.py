"""A linear layer on 8-bit integers and its quantiser (include/i8_linear.h).

A quantised matrix is a pair (q, scale): q in torch.int8 and one FP32 scale for each row, so that
element (i, j) stands for q[i, j] * scale[i]. Activations have a scale for each token, weights
(outputs, inputs) one for each output channel:
    q, s = i8_quantize(x);  wq, ws = i8_quantize(w);  y = i8_linear(q, s, wq, ws, bias)
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import I8_EXPORTED, SgemmError, _on_stream, lib
from .f8 import _TYPE, _rows, _stream_here

__all__ = ["i8_quantize", "i8_linear", "i8_linear_plan", "i8_linear_status", "I8_EXPORTED"]

# i8_quantize_args and i8_linear_args
_quantize_args = struct.Struct("@iiPiiPiPP").pack
_linear_args = struct.Struct("@iiiPiPPiPPfPiiP").pack


def i8_quantize(x, *, stream=None):
    """Quantise the rows of a 2-D CUDA tensor (float32, bfloat16, float16): returns (q, scale), with
    scale = a / 127 for the row's largest magnitude a, and q = x * (127 / a) rounded to whole numbers.
    `stream`: where to run (a torch stream or a handle; the current stream unless given), the results
    belong to it."""
    if stream is not None:
        return _on_stream(stream, lambda: i8_quantize(x), (x,))
    kind = _TYPE.get(x.dtype)
    if kind is None:
        raise TypeError("x must be float32, bfloat16 or float16")
    rows, cols, ldx = _rows("x", x)
    _, handle = _stream_here("x", x)
    device = x.device
    # rows of a multiple of 16 bytes, as the product's copies need them
    ldq = (cols + 15) // 16 * 16 or 1
    q = torch.empty_strided((rows, cols), (ldq, 1), dtype=torch.int8, device=device)
    scale = torch.empty(rows, dtype=torch.float32, device=device)
    rc = lib.i8_quantize_with(_quantize_args(rows, cols, x.data_ptr(), kind, ldx, q.data_ptr(), ldq,
                                             scale.data_ptr(), handle))
    if rc != 0:
        raise SgemmError(rc, "i8_quantize")
    return q, scale


def _operand(name, q, scale):
    """(rows, columns, row stride) of a quantised matrix."""
    if q.dtype is not torch.int8:
        raise TypeError(f"{name} must be int8")
    rows, cols, ld = _rows(name, q)
    if rows <= 1 or cols == 0:  # (nothing is read from row to row)
        ld = (ld + 15) // 16 * 16
    if scale.dtype is not torch.float32:
        raise TypeError(f"{name}'s scale must be a float32 CUDA tensor")
    if scale.shape != (rows,) or not scale.is_contiguous():
        raise ValueError(f"{name}'s scale must be a contiguous vector with one entry for each row")
    return rows, cols, ld


def i8_linear(x, x_scale, w, w_scale, bias=None, *, beta=0.0, out=None, out_dtype=None, stream=None):
    """out = x @ w^T + bias + beta * out on quantised matrices x (tokens, inputs) and w (outputs,
    inputs). The sums over the inputs are exact whole numbers, scales, bias (float32) and beta are
    applied in float32 with one rounding to out's type. `out` is float32, bfloat16 or float16 with unit
    column stride; without one a new tensor of out_dtype (bfloat16 unless given) is returned. `stream`
    as in i8_quantize. Raises SgemmError on a nonzero status."""
    if stream is not None:
        return _on_stream(stream, lambda: i8_linear(
            x, x_scale, w, w_scale, bias, beta=beta, out=out, out_dtype=out_dtype),
            [t for t in (x, x_scale, w, w_scale, bias, out) if t is not None])
    M, K, ldx = _operand("x", x, x_scale)
    N, K2, ldw = _operand("w", w, w_scale)
    if K2 != K:
        raise ValueError("shape mismatch")
    at, handle = _stream_here("x", x)
    bp = 0
    if bias is not None:
        if bias.dtype is not torch.float32:
            raise TypeError("bias must be float32")
        if bias.shape != (N,) or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous vector of {N} elements")
        if bias.get_device() != at:
            raise ValueError("bias is on another device")
        bp = bias.data_ptr()
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs an out to scale")
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=x.device)
        ldd = N or 1
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out has another type than out_dtype")
        rows, cols, ldd = _rows("out", out)
        if rows != M or cols != N:
            raise ValueError("shape mismatch")
    kind = _TYPE.get(out.dtype)
    if kind is None:
        raise TypeError("out must be float32, bfloat16 or float16")
    if not (at == w.get_device() == out.get_device() == x_scale.get_device() == w_scale.get_device()):
        raise ValueError("operands, scales and out must be on one device")
    rc = lib.i8_linear_with(_linear_args(
        M, N, K, x.data_ptr(), ldx, x_scale.data_ptr(), w.data_ptr(), ldw, w_scale.data_ptr(), bp, beta,
        out.data_ptr(), kind, ldd, handle))
    if rc != 0:
        raise SgemmError(rc, "i8_linear")
    return out


def i8_linear_plan(M, N, K, num_sms=0) -> dict:
    """How i8_linear runs a product: {"tile_tokens", "tile_channels", "split"} (see the header)."""
    v = [ctypes.c_int(0) for _ in range(3)]
    rc = lib.i8_linear_plan(M, N, K, num_sms, *[ctypes.byref(x) for x in v])
    if rc != 0:
        raise SgemmError(rc, "i8_linear_plan")
    return {"tile_tokens": v[0].value, "tile_channels": v[1].value, "split": v[2].value}


def i8_linear_status() -> tuple[int, int]:
    """(call status, device status word of i8_linear); reading clears the word."""
    v = ctypes.c_int(0)
    rc = lib.i8_linear_status(ctypes.byref(v))
    return rc, v.value
