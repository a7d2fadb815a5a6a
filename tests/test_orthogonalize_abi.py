"""CPU-only checks of the orthogonalisation's C ABI: exported symbols, refusals of illegal
arguments (before any CUDA call) and the workspace query."""
import ctypes
import os
import re

import pytest
import torch

import dense_fp32_matrix_08_gb300 as sg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "orthogonalize.h")
P = 1 << 20  # never dereferenced
USUAL = (ctypes.c_float * 3)(3.4445, -4.7750, 2.0315)


def test_every_declared_symbol_is_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(sg.NS_EXPORTED)
    for n in names:
        assert hasattr(sg.lib, n)


CALL = dict(batch=2, rows=4, cols=6, G=P, gt=0, ldg=6, gs=24, steps=5, co=USUAL, eps=1e-7,
            alpha=1.0, beta=0.0, out=P, ot=0, ldo=6, os=24)


def coefficients(*v):
    return (ctypes.c_float * 3)(*v)


@pytest.mark.parametrize("change,code", [
    (dict(batch=-1), -1), (dict(rows=-1), -2), (dict(cols=-1), -3), (dict(G=None), -4),
    (dict(G=P + 2), -4), (dict(gt=1, G=P + 1), -4), (dict(gt=3), -5), (dict(ldg=5), -6),
    (dict(gs=-1), -7), (dict(steps=-1), -8), (dict(steps=65), -8), (dict(co=None), -9),
    (dict(co=coefficients(float("inf"), 0, 0)), -9), (dict(co=coefficients(1e8, 0, 0)), -9),
    (dict(eps=-1e-9), -10), (dict(eps=float("nan")), -10), (dict(out=None), -13),
    (dict(out=P + 1), -13), (dict(ot=-1), -14), (dict(ldo=5), -15), (dict(os=-1), -16),
    (dict(os=23), -16),  # results of two matrices would overlap
    (dict(batch=-1, rows=-1, G=None), -1),
])
def test_illegal_arguments(change, code):
    assert sg.lib.ns_orthogonalize(*{**CALL, **change}.values(), None) == code


def test_empty_needs_no_pointers():
    for change in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert sg.lib.ns_orthogonalize(*{**CALL, "G": None, "out": None, **change}.values(), None) == 0


def test_workspace_size():
    assert sg.ns_orthogonalize_workspace_size(-1, 4, 4)[0] == -1
    assert sg.ns_orthogonalize_workspace_size(1, -4, 4)[0] == -2
    assert sg.ns_orthogonalize_workspace_size(1, 4, -4)[0] == -3
    assert sg.ns_orthogonalize_workspace_size(1, 0, 4) == (0, 0)
    rc, wide = sg.ns_orthogonalize_workspace_size(1, 300, 1000)
    assert rc == 0 and wide > 2 * 4 * 300 * 1000  # two X as pairs of FP16 numbers
    assert sg.ns_orthogonalize_workspace_size(1, 1000, 300) == (0, wide)
    assert sg.ns_orthogonalize_workspace_size(3, 300, 1000)[1] > 2 * wide


def test_python_refusals():
    with pytest.raises(TypeError):  # not on a CUDA device
        sg.orthogonalize(torch.zeros(3, 3))
    with pytest.raises(ValueError):
        sg.orthogonalize(torch.zeros(3))
    with pytest.raises(TypeError):
        sg.orthogonalize(torch.zeros(3, 3, dtype=torch.int32))
