"""CPU-only checks of the C ABI of the linear layer on 8-bit integers and of its Python entry points:
exported symbols, refusals of illegal arguments, which come before any CUDA call, plans, and the bounded
waits of the kernel's source."""
import os
import random
import re

import pytest
import torch

import dense_fp32_matrix_08_gb300 as sg
from i8_plans import SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a 16-byte aligned address that is never dereferenced


def test_every_declared_symbol_is_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "i8_linear.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(sg.I8_EXPORTED)
    for n in names:
        assert hasattr(sg.lib, n)


QUANT = dict(rows=4, cols=8, x=P, xt=0, ldx=8, q=P, ldq=8, s=P)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), -1), (dict(cols=-1), -2), (dict(x=None), -3), (dict(x=P + 2), -3), (dict(xt=1, x=P + 1), -3),
    (dict(xt=3), -4), (dict(ldx=7), -5), (dict(cols=0, ldx=0), -5), (dict(q=None), -6), (dict(ldq=7), -7),
    (dict(s=None), -8), (dict(cols=0, s=None), -8),
])
def test_quantize_illegal_arguments(change, code):
    assert sg.lib.i8_quantize(*{**QUANT, **change}.values(), None) == code


def test_quantize_of_no_rows_needs_no_pointers():
    assert sg.lib.i8_quantize(*{**QUANT, "rows": 0, "x": None, "q": None, "s": None}.values(), None) == 0


LINEAR = dict(M=4, N=8, K=20, x=P, ldx=32, sx=P, w=P, ldw=32, sw=P, bias=None, beta=0.0, D=P, dt=0, ldd=8)


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), -1), (dict(N=-1), -2), (dict(K=-1), -3), (dict(K=131072, ldx=131072, ldw=131072), -3),
    (dict(x=None), -4), (dict(x=P + 8), -4), (dict(ldx=16), -5), (dict(ldx=24), -5), (dict(K=0, ldx=0), -5),
    (dict(sx=None), -6), (dict(w=None), -7), (dict(w=P + 4), -7), (dict(ldw=16), -8), (dict(ldw=33), -8),
    (dict(sw=None), -9), (dict(D=None), -12), (dict(D=P + 2), -12), (dict(dt=1, D=P + 1), -12), (dict(dt=3), -13),
    (dict(ldd=7), -14), (dict(M=-1, N=-1, D=None), -1),
])
def test_linear_illegal_arguments(change, code):
    assert sg.lib.i8_linear(*{**LINEAR, **change}.values(), None) == code


def test_empty_product_needs_no_pointers():
    none = dict(x=None, sx=None, w=None, sw=None, D=None)
    assert sg.lib.i8_linear(*{**LINEAR, **none, "M": 0}.values(), None) == 0
    assert sg.lib.i8_linear(*{**LINEAR, **none, "N": 0}.values(), None) == 0
    assert sg.lib.i8_linear_with(None) == -1 and sg.lib.i8_quantize_with(None) == -1


def test_plans():
    for M, N, K, code in ((0, 1, 1, -1), (1, 0, 1, -2), (1, 1, 0, -3), (1, 1, 131072, -3)):
        assert sg.lib.i8_linear_plan(M, N, K, 152, None, None, None) == code
    assert sg.lib.i8_linear_plan(1, 1, 1, -1, None, None, None) == -4
    assert sg.i8_linear_plan(1, 4096, 4096, 152) == {"tile_tokens": 0, "tile_channels": 0, "split": 1}
    assert sg.i8_linear_plan(8192, 14336, 4096, 152) == {"tile_tokens": 128, "tile_channels": 256, "split": 1}
    for M in (3, 16, 40, 100, 500, 5000):
        for N in (1, 300, 4096):
            for K in (1, 700, 131071):
                plan = sg.i8_linear_plan(M, N, K, 152)
                blocks = -(-K // 128)
                assert plan["tile_tokens"] in (16, 32, 64, 128) and plan["split"] in (1, 2, 4, 8)
                assert plan["tile_channels"] == 128 or plan["tile_tokens"] == 128
                assert plan["split"] <= blocks and (plan["split"] == 1 or plan["tile_channels"] == 128)


def test_every_plan_has_a_shape():
    """The listed shapes run as they say, and a search finds no other way to run."""
    for plan, shape in SHAPES.items():
        assert tuple(sg.i8_linear_plan(*shape, 152).values()) == plan
    r = random.Random(3)
    found = {tuple(sg.i8_linear_plan(*(min(131071, int(2 ** r.uniform(0, top))) for top in (13.5, 14.5, 17)), 152)
                   .values()) for _ in range(20000)}
    assert found <= set(SHAPES), found - set(SHAPES)


def test_warps_leave_their_waits_together():
    """When a bounded wait runs out while its phase completes, some lanes are told so and others are
    not: the answer has to be the warp's, a vote on it. (Making it happen would need a wait that runs
    out at a chosen moment, so this reads the source.)"""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(ROOT, "dense_fp32_matrix_08_gb300", "csrc",
                                                     "i8_linear.cu")).read())
    statements = [" ".join(s.split()) for s in re.split(r"[;{}]", text) if "wait_short(" in s]
    assert len(statements) >= 5
    for s in statements:
        # (a wait whose answer nothing depends on: copies that must land before the warp leaves)
        assert re.search(r"__all_sync\(0xffffffffu, .*wait_short\(", s) or re.fullmatch(
            r"(if \(!PAIR \|\| cta == 0\) )?wait_short\([^;]*\)", s), s


def test_python_refusals():
    x = torch.zeros(4, 16)
    q, s = torch.zeros(4, 16, dtype=torch.int8), torch.ones(4)
    with pytest.raises(TypeError):
        sg.i8_quantize(x.double())
    with pytest.raises(TypeError):  # not on a CUDA device
        sg.i8_quantize(x)
    with pytest.raises(ValueError):
        sg.i8_quantize(x[0])
    with pytest.raises(TypeError):
        sg.i8_linear(x, s, q, s)
    with pytest.raises(TypeError):
        sg.i8_linear(q, s, q, s)
