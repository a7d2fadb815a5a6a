"""CPU-only checks of the 8-bit operators' C ABI and of their Python entry points: exported
symbols and refusals of illegal arguments, which come before any CUDA call."""
import os
import re

import pytest
import torch

import dense_fp32_matrix_08_gb300 as sg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "f8_gemm.h")
P = 1 << 20  # a 16-byte aligned address that is never dereferenced


def test_every_declared_symbol_is_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(sg.F8_EXPORTED)
    for n in names:
        assert hasattr(sg.lib, n)


GEMM = dict(transa=0, transb=0, M=4, N=4, K=4, alpha=1.0, A=P, af=0, lda=16, sa=P, ar=1, sam=1,
            sak=1, B=P, bf=0, ldb=16, sb=P, bc=128, sbm=1, sbk=1, beta=0.0, D=P, dt=0, ldd=4)


@pytest.mark.parametrize("change,code", [
    (dict(transa=2), -1), (dict(transb=-1), -2), (dict(M=-1), -3), (dict(N=-1), -4),
    (dict(K=-1), -5), (dict(A=None), -7), (dict(A=P + 8), -7), (dict(af=2), -8),
    (dict(lda=8), -9), (dict(lda=20), -9), (dict(lda=16, K=17), -9),
    (dict(transa=1, M=17), -9), (dict(sa=None), -10), (dict(ar=64), -11), (dict(sam=-1), -12),
    (dict(sak=-1), -13), (dict(B=None), -14), (dict(B=P + 1), -14), (dict(bf=-1), -15),
    (dict(ldb=0), -16), (dict(N=17, ldd=17), -16), (dict(transb=1, K=17, lda=32), -16),
    (dict(sb=None), -17), (dict(bc=0), -18), (dict(sbm=-1), -19), (dict(sbk=-1), -20),
    (dict(D=None), -22), (dict(D=P + 2), -22), (dict(dt=1, D=P + 1), -22), (dict(dt=3), -23),
    (dict(ldd=3), -24),
    (dict(M=-1, N=-1, D=None), -3),  # the first illegal one
])
def test_gemm_illegal_arguments(change, code):
    assert sg.lib.f8_gemm(*{**GEMM, **change}.values(), None) == code


def test_gemm_empty_needs_no_pointers():
    none = dict(A=None, B=None, sa=None, sb=None, D=None)
    assert sg.lib.f8_gemm(*{**GEMM, **none, "M": 0}.values(), None) == 0
    assert sg.lib.f8_gemm(*{**GEMM, **none, "N": 0}.values(), None) == 0


QUANT = dict(rows=4, cols=4, x=P, xt=0, ldx=4, br=1, bc=128, fmt=0, pow2=0, q=P, ldq=4, s=P,
             srow=1, scol=1, qc=None, ldqc=0, sc=None, scr=0, scc=0)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), -1), (dict(cols=-1), -2), (dict(x=None), -3), (dict(x=P + 2), -3),
    (dict(xt=5), -4), (dict(ldx=3), -5), (dict(br=2), -6), (dict(bc=64), -7),
    (dict(br=1, bc=1), -7), (dict(fmt=7), -8), (dict(q=None), -10), (dict(ldq=3), -11),
    (dict(s=None), -12), (dict(srow=-1), -13), (dict(scol=-1), -14),
    (dict(br=128, qc=P, ldqc=4, sc=P), -15), (dict(qc=P, ldqc=3, sc=P), -16),
    (dict(qc=P, ldqc=4), -17), (dict(qc=P, ldqc=4, sc=P, scr=-1), -18),
    (dict(qc=P, ldqc=4, sc=P, scc=-1), -19),
])
def test_quantize_illegal_arguments(change, code):
    assert sg.lib.f8_quantize(*{**QUANT, **change}.values(), None) == code


def test_quantize_empty_needs_no_pointers():
    none = dict(x=None, q=None, s=None)
    assert sg.lib.f8_quantize(*{**QUANT, **none, "rows": 0}.values(), None) == 0
    assert sg.lib.f8_quantize(*{**QUANT, **none, "cols": 0}.values(), None) == 0


def test_python_refusals():
    x = torch.zeros(4, 4)
    q = torch.zeros(4, 16, dtype=torch.float8_e4m3fn)
    s = torch.ones(4, 1)
    with pytest.raises(ValueError):
        sg.f8_quantize(x, (64, 64))
    with pytest.raises(TypeError):
        sg.f8_quantize(x, dtype=torch.int8)
    with pytest.raises(TypeError):
        sg.f8_quantize(x.double())
    with pytest.raises(TypeError):  # not on a CUDA device
        sg.f8_quantize(x)
    with pytest.raises(ValueError):
        sg.f8_quantize(x[0])
    with pytest.raises(TypeError):
        sg.f8_matmul(x, s, q, s)
    with pytest.raises(TypeError):
        sg.f8_matmul(q, s, q, s, transb=True)
