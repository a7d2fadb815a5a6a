"""8-bit block-scaled products and their quantiser (include/f8_gemm.h).

A quantised matrix is a pair (q, scale): q in torch.float8_e4m3fn or torch.float8_e5m2 and FP32
scales, one for each block of 1 x 128, 128 x 1 or 128 x 128 elements of q, so that element (i, j)
stands for q[i, j] * scale[i // block_rows, j // block_cols]. `scale` has one entry for each
block; its shape tells the block shape.

For a linear layer y = x W^T:
    forward          x (1, 128), W (128, 128):   f8_matmul(xq, xs, wq, ws, transb=True)
    input gradient   dy (1, 128), W (128, 128):  f8_matmul(dyq, dys, wq, ws)
    weight gradient  dy, x (128, 1):             f8_matmul(dyc, dycs, xc, xcs, transa=True)
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import F8_EXPORTED, SgemmError, _on_stream, _stream, lib

__all__ = ["f8_quantize", "f8_quantize_pair", "f8_matmul", "f8_gemm_plan", "f8_gemm_status",
           "F8_EXPORTED"]

_FORMAT = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
_TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_MOST = 0x7ffffff0  # sizes are 32-bit, rows of quantised matrices multiples of 16
_BLOCKS = ((1, 128), (128, 1), (128, 128))

# f8_quantize_args and f8_gemm_args
_quantize_args = struct.Struct("@iiPiiiiiiPiPqqPiPqqP").pack
_gemm_args = struct.Struct("@iiiiifPiiPiqqPiiPiqqfPiiP").pack


def _rows(name, t):
    """(rows, columns, row stride) of a 2-D CUDA tensor with unit column stride and rows that do not
    overlap."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise TypeError(f"{name} must live on a CUDA device")
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows <= 1:
        ld = cols
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap (an expanded tensor or a sliding window)")
    if rows > _MOST or ld > _MOST:
        raise ValueError(f"{name}'s sizes and row stride must be below 2^31 - 15")
    return rows, cols, ld or 1


def _quantize(x, block, both, dtype, pow2, stream):
    if stream is not None:
        return _on_stream(stream, lambda: _quantize(x, block, both, dtype, pow2, None), (x,))
    fmt = _FORMAT.get(dtype)
    if fmt is None:
        raise TypeError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2")
    xt = _TYPE.get(x.dtype)
    if xt is None:
        raise TypeError("x must be float32, bfloat16 or float16")
    rows, cols, ldx = _rows("x", x)
    device = x.device
    br, bc = block
    ldq = (cols + 15) // 16 * 16 or 1
    nb = (cols + 127) >> 7
    # rows of a multiple of 16 bytes, as the product's copies need them
    q = torch.empty_strided((rows, cols), (ldq, 1), dtype=dtype, device=device)
    if br == 1:
        # neighbouring rows' scales of one block are neighbours, as the product reads them
        s_row, s_col = 1, rows or 1
        s = torch.empty_strided((rows, nb), (1, s_col), dtype=torch.float32, device=device)
    else:
        s_row, s_col = (cols if bc == 1 else nb) or 1, 1
        s = torch.empty_strided(((rows + 127) >> 7, cols if bc == 1 else nb), (s_row, 1),
                                dtype=torch.float32, device=device)
    if both:
        qc = torch.empty_strided((rows, cols), (ldq, 1), dtype=dtype, device=device)
        sc = torch.empty_strided(((rows + 127) >> 7, cols), (cols or 1, 1), dtype=torch.float32,
                                 device=device)
        rc = lib.f8_quantize_with(_quantize_args(
            rows, cols, x.data_ptr(), xt, ldx, br, bc, fmt, pow2, q.data_ptr(), ldq, s.data_ptr(),
            s_row, s_col, qc.data_ptr(), ldq, sc.data_ptr(), cols, 1, _stream(None) or 0))
    else:
        rc = lib.f8_quantize_with(_quantize_args(
            rows, cols, x.data_ptr(), xt, ldx, br, bc, fmt, pow2, q.data_ptr(), ldq, s.data_ptr(),
            s_row, s_col, 0, 0, 0, 0, 0, _stream(None) or 0))
    if rc != 0:
        raise SgemmError(rc, "f8_quantize")
    return (q, s, qc, sc) if both else (q, s)


def f8_quantize(x, block=(1, 128), *, dtype=torch.float8_e4m3fn, pow2=False, stream=None):
    """Quantise a 2-D CUDA tensor (float32, bfloat16, float16) by blocks of (1, 128), (128, 1) or
    (128, 128): returns (q, scale). scale = max(amax / largest, 2^-126) of each block, with pow2
    the least power of two not below it; q = x / scale rounded to dtype. `stream`: where to run (a
    torch stream or a handle; the current stream unless given), the results belong to it."""
    if block not in _BLOCKS:
        raise ValueError(f"block must be one of {_BLOCKS}")
    return _quantize(x, block, False, dtype, bool(pow2), stream)


def f8_quantize_pair(x, *, dtype=torch.float8_e4m3fn, pow2=False, stream=None):
    """f8_quantize by (1, 128) and by (128, 1) blocks from one read of x: returns
    (q_rows, scale_rows, q_columns, scale_columns)."""
    return _quantize(x, (1, 128), True, dtype, bool(pow2), stream)


def _operand(name, q, scale, k_dim):
    """(format, ld, group, stride along the other dimension, stride along k, k, other size) of an
    operand."""
    fmt = _FORMAT.get(q.dtype)
    if fmt is None:
        raise TypeError(f"{name} must be torch.float8_e4m3fn or torch.float8_e5m2")
    rows, cols, ld = _rows(name, q)
    if rows <= 1:
        ld = (ld + 15) // 16 * 16
    if scale.dtype is not torch.float32 or scale.dim() != 2 or not scale.is_cuda:
        raise TypeError(f"{name}'s scale must be a 2-D float32 CUDA tensor")
    if k_dim:
        mn, k = rows, cols
        have, blocks = scale.shape
        s_mn, s_k = scale.stride()
    else:
        k, mn = rows, cols
        blocks, have = scale.shape
        s_k, s_mn = scale.stride()
    if blocks != (k + 127) >> 7:
        raise ValueError(f"{name}'s scale needs one entry for each 128 along the contraction")
    if have == mn:
        return fmt, ld, 1, s_mn, s_k, k, mn
    if have == (mn + 127) >> 7:
        return fmt, ld, 128, s_mn, s_k, k, mn
    raise ValueError(f"{name}'s scale does not fit its shape")


def f8_matmul(a, a_scale, b, b_scale, *, transa=False, transb=False, alpha=1.0, beta=0.0,
              out=None, out_dtype=None, stream=None):
    """out = alpha * op(a) @ op(b) + beta * out on quantised operands (op: transposed if the
    flag is set). `out` is float32, bfloat16 or float16 with unit column stride; without one a
    new tensor of out_dtype (bfloat16 unless given) is returned. Each operand's scales run along
    the contraction in blocks of 128. `stream` as in f8_quantize. Raises SgemmError on a nonzero
    status."""
    if stream is not None:
        return _on_stream(stream, lambda: f8_matmul(
            a, a_scale, b, b_scale, transa=transa, transb=transb, alpha=alpha, beta=beta, out=out,
            out_dtype=out_dtype), [t for t in (a, a_scale, b, b_scale, out) if t is not None])
    fa, lda, ga, amn, ak, K, M = _operand("a", a, a_scale, 0 if transa else 1)
    fb, ldb, gb, bmn, bk, K2, N = _operand("b", b, b_scale, 1 if transb else 0)
    if K2 != K:
        raise ValueError("shape mismatch")
    device = a.device
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs an out to scale")
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=device)
        ldd = N or 1
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out has another type than out_dtype")
        rows, cols, ldd = _rows("out", out)
        if rows != M or cols != N:
            raise ValueError("shape mismatch")
    dt = _TYPE.get(out.dtype)
    if dt is None:
        raise TypeError("out must be float32, bfloat16 or float16")
    if not (device == b.device == out.device == a_scale.device == b_scale.device):
        raise ValueError("operands, scales and out must be on one device")
    rc = lib.f8_gemm_with(_gemm_args(
        transa, transb, M, N, K, alpha, a.data_ptr(), fa, lda, a_scale.data_ptr(), ga, amn, ak,
        b.data_ptr(), fb, ldb, b_scale.data_ptr(), gb, bmn, bk, beta, out.data_ptr(), dt, ldd,
        _stream(None) or 0))
    if rc != 0:
        raise SgemmError(rc, "f8_gemm")
    return out


def f8_gemm_plan(M, N, K, *, transa=False, transb=False, a_rows=1, b_cols=128, num_sms=0) -> dict:
    """How f8_matmul runs a product: {"exchanged", "tile_cols", "split"} (see the header); a_rows and
    b_cols are the rows of op(a) and the columns of op(b) that share a scale."""
    v = [ctypes.c_int(0) for _ in range(3)]
    rc = lib.f8_gemm_plan(int(transa), int(transb), M, N, K, a_rows, b_cols, num_sms,
                          *[ctypes.byref(x) for x in v])
    if rc != 0:
        raise SgemmError(rc, "f8_gemm_plan")
    return {"exchanged": bool(v[0].value), "tile_cols": v[1].value, "split": v[2].value}


def f8_gemm_status() -> tuple[int, int]:
    """(call status, device status word of f8_gemm); reading clears the word."""
    v = ctypes.c_int(0)
    rc = lib.f8_gemm_status(ctypes.byref(v))
    return rc, v.value
