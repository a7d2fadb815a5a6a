"""CPU-only checks of the C ABI of layer norm and of clipping, and of their Python entry points:
exported symbols and refusals of illegal arguments, which come before any CUDA call."""
import ctypes
import os
import re

import pytest
import torch

import dense_fp32_matrix_08_gb300 as sg

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
P = 1 << 20  # a 16-byte aligned address that is never dereferenced


@pytest.mark.parametrize("header,names", [("layer_norm.h", sg.LN_EXPORTED), ("grad_clip.h", sg.GC_EXPORTED)])
def test_every_declared_symbol_is_bound(header, names):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    assert set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)) == set(names)
    for n in names:
        assert hasattr(sg.lib, n)


NORM = dict(rows=4, cols=8, x=P, xt=0, ldx=8, w=P, b=P, wt=0, eps=1e-5, y=P, ldy=8, mean=P, rstd=P)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), -1), (dict(cols=0), -2), (dict(cols=-1), -2), (dict(x=None), -3), (dict(x=P + 2), -3),
    (dict(xt=1, x=P + 1), -3), (dict(xt=3), -4), (dict(ldx=7), -5), (dict(w=P + 2), -6), (dict(b=P + 1), -7),
    (dict(wt=-1), -8), (dict(eps=-1e-9), -9), (dict(eps=float("nan")), -9), (dict(eps=float("inf")), -9),
    (dict(y=None), -10), (dict(y=P + 3), -10), (dict(ldy=0), -11), (dict(rows=-1, cols=0, y=None), -1),
])
def test_norm_illegal_arguments(change, code):
    assert sg.lib.layer_norm(*{**NORM, **change}.values(), None) == code


def test_norm_without_rows_needs_no_pointers():
    none = dict(rows=0, x=None, w=None, b=None, y=None, mean=None, rstd=None)
    assert sg.lib.layer_norm(*{**NORM, **none}.values(), None) == 0


BACK = dict(rows=4, cols=8, dy=P, lddy=8, x=P, xt=0, ldx=8, mean=P, rstd=P, w=P, wt=0, dx=P, lddx=8, dw=P, db=P,
            beta=0.0)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), -1), (dict(cols=0), -2), (dict(dy=None), -3), (dict(dy=P + 2), -3), (dict(lddy=7), -4),
    (dict(x=None), -5), (dict(x=P + 1), -5), (dict(xt=9), -6), (dict(ldx=3), -7), (dict(mean=None), -8),
    (dict(rstd=None), -9), (dict(w=P + 2), -10), (dict(wt=3), -11), (dict(dx=P + 2), -12), (dict(lddx=7), -13),
])
def test_backward_illegal_arguments(change, code):
    assert sg.lib.layer_norm_backward(*{**BACK, **change}.values(), None) == code


def test_backward_with_nothing_to_do():
    none = dict(rows=0, dy=None, x=None, mean=None, rstd=None, w=None, dx=None)
    assert sg.lib.layer_norm_backward(*{**BACK, **none, "beta": 1.0}.values(), None) == 0
    assert sg.lib.layer_norm_backward(*{**BACK, "dx": None, "dw": None, "db": None}.values(), None) == 0


def test_missing_structures_and_workspace():
    assert sg.lib.layer_norm_with(None) == -1 and sg.lib.layer_norm_backward_with(None) == -1
    n = ctypes.c_size_t(1)
    assert sg.lib.layer_norm_backward_workspace_size(-1, 4, ctypes.byref(n)) == -1
    assert sg.lib.layer_norm_backward_workspace_size(4, 0, None) == -2
    assert sg.layer_norm_backward_workspace_size(0, 4) == (0, 0)
    for rows, cols in ((1, 1), (8192, 4096), (5, 100000), (1 << 30, 8), (1, (1 << 31) - 1)):
        rc, size = sg.layer_norm_backward_workspace_size(rows, cols)
        assert rc == 0 and size >= 8 * cols
        assert size <= 8 * cols * (rows // 512 + 16 * 608 + 1) + 16 * rows + 256


def arrays(count, at, types, sizes):
    return ((ctypes.c_void_p * max(1, count))(*at), (ctypes.c_int * max(1, count))(*types),
            (ctypes.c_longlong * max(1, count))(*sizes))


def clip(at=(P, 2 * P), types=(0, 1), sizes=(10, 20), max_norm=1.0, eps=1e-6, out="same", out_types=None,
         count=None, norm=P, **none):
    g, t, n = arrays(len(at), at, types, sizes)
    o = None
    if out is not None:
        o, ot, _ = arrays(len(at), at if out == "same" else out, out_types or types, sizes)
    return sg.lib.clip_grad_norm(len(at) if count is None else count, none.get("g", g), none.get("t", t),
                                 none.get("n", n), max_norm, eps, o,
                                 none.get("ot", ot if out is not None else None), norm, None)


@pytest.mark.parametrize("change,code", [
    (dict(count=-1), -1), (dict(g=None), -2), (dict(at=(P, 0)), -2), (dict(at=(P + 2, 2 * P)), -2),
    (dict(at=(P, 2 * P + 1)), -2), (dict(t=None), -3), (dict(types=(0, 3)), -3), (dict(n=None), -4),
    (dict(sizes=(10, -1)), -4), (dict(max_norm=-1.0), -5), (dict(max_norm=float("nan")), -5),
    (dict(eps=-1.0), -6), (dict(eps=float("inf")), -6), (dict(eps=float("nan")), -6),
    (dict(out=(P, 0)), -7), (dict(out=(P, 2 * P + 1)), -7), (dict(out=(P + 4, 2 * P)), -7),
    (dict(at=(P, P + 39), types=(0, 0)), -2), (dict(at=(P, P + 36), types=(0, 0)), -7),
    (dict(at=(P, P)), -7), (dict(out=(2 * P, 3 * P)), -7), (dict(out=(3 * P, 3 * P + 36), out_types=(0, 0)), -7),
    (dict(out=(P, 3 * P), out_types=(1, 1)), -7),  # another type in place
    (dict(out=(P, 2 * P), out_types=(0, 7)), -8), (dict(ot=None), -8),
])
def test_clip_illegal_arguments(change, code):
    assert clip(**change) == code


def test_clip_of_nothing():
    assert clip(at=(), types=(), sizes=(), norm=None) == 0
    assert clip(at=(0, 0), sizes=(0, 0), norm=None) == 0  # empty arrays need no address


def test_overlaps_are_found_by_address_and_not_by_order():
    def refused(spans, outs):
        at, sizes = zip(*spans)
        return clip(at=at, types=[0] * len(at), sizes=sizes, out=outs) == -7

    a, n = P, 256  # 64 elements
    assert refused([(a, 64), (a + n - 4, 64)], (a, a + n - 4))
    assert refused([(a + n - 4, 64), (a, 64)], (a + n - 4, a))
    assert refused([(a, 1000), (a + 8, 1)], (a + 8000, a + 9000))
    assert refused([(a, 64), (a, 64), (a, 64)], (a, a + n, a + 2 * n))
    assert refused([(a, 64), (a + n, 64)], (a + 10 * n, a))


def test_python_refusals():
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        sg.layer_norm(x.double())
    with pytest.raises(TypeError):  # not on a CUDA device
        sg.layer_norm(x)
    with pytest.raises(ValueError):
        sg.layer_norm(x[0])
    with pytest.raises(TypeError):
        sg.layer_norm_backward(x, x, x[:, 0], x[:, 0])
    with pytest.raises(TypeError):
        sg.clip_grad_norm([x], 1.0)
    with pytest.raises(TypeError):
        sg.clip_grad_norm([3.0], 1.0)
