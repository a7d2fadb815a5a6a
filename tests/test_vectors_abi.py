"""CPU-only: vectors of FP32 numbers that are not aligned to their elements are refused with their own
argument's number before any CUDA call. (On the GPU such an access would be misaligned.)"""
import pytest

import dense_fp32_matrix_08_gb300 as sg
from test_f8_abi import GEMM, QUANT as F8_QUANT
from test_i8_abi import LINEAR, QUANT
from test_norm_clip_abi import BACK, NORM, P, clip

ODD = [P + 1, P + 2, P + 3]


@pytest.mark.parametrize("at", ODD)
@pytest.mark.parametrize("call,args,change,code", [
    ("layer_norm", NORM, "mean", -12), ("layer_norm", NORM, "rstd", -13),
    ("layer_norm_backward", BACK, "mean", -8), ("layer_norm_backward", BACK, "rstd", -9),
    ("layer_norm_backward", BACK, "dw", -14), ("layer_norm_backward", BACK, "db", -15),
    ("i8_quantize", QUANT, "s", -8),
    ("i8_linear", LINEAR, "sx", -6), ("i8_linear", LINEAR, "sw", -9), ("i8_linear", LINEAR, "bias", -10),
])
def test_refused(call, args, change, code, at):
    assert getattr(sg.lib, call)(*{**args, change: at}.values(), None) == code


@pytest.mark.parametrize("at", ODD)
def test_norm_of_gradients_refused(at):
    assert clip(norm=at) == -9
    assert clip(norm=at, out=None) == -9
    assert clip(norm=at, out=(P, 0)) == -7  # the first illegal one


def test_the_first_illegal_argument_is_told():
    assert sg.lib.layer_norm(*{**NORM, "ldy": 7, "mean": P + 1}.values(), None) == -11
    assert sg.lib.layer_norm_backward(*{**BACK, "rstd": P + 1, "w": P + 2}.values(), None) == -9
    assert sg.lib.layer_norm_backward(*{**BACK, "lddx": 7, "dw": P + 1}.values(), None) == -13
    assert sg.lib.i8_linear(*{**LINEAR, "bias": P + 2, "D": None}.values(), None) == -10


@pytest.mark.parametrize("at", ODD)
@pytest.mark.parametrize("call,args,change,code", [
    ("f8_gemm", GEMM, dict(sa=0), -10), ("f8_gemm", GEMM, dict(sb=0), -17),
    ("f8_quantize", F8_QUANT, dict(s=0), -12),
    ("f8_quantize", F8_QUANT, dict(qc=P, ldqc=4, sc=0, scr=1, scc=1), -17),
])
def test_scales_of_the_8_bit_product_refused(call, args, change, code, at):
    change = {k: at if v == 0 else v for k, v in change.items()}
    assert getattr(sg.lib, call)(*{**args, **change}.values(), None) == code
