"""GPU tests of layer norm and its gradients in place in every layout of a row, with several rows for each block, and
of parameters at any alignment: where things lie changes no bit of a result."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

from test_gpu_layer_norm import TYPES, check, problem

COLS = [40, 250, 512, 1000, 2000, 4096, 5000, 8192, 12288, 16384, 17000]


def at_any(t, offset):
    """A copy of t in rows that begin `offset` elements after a 16-byte boundary."""
    pitch = (t.shape[1] + offset + 7) // 8 * 8
    return torch.zeros(t.shape[0], pitch, dtype=t.dtype, device="cuda")[:, offset:offset + t.shape[1]].copy_(t)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_in_place(cols, dtype, offset):
    x, w, b, dy = problem(460, cols, dtype)
    x, dy = at_any(x, offset), at_any(dy, offset)
    y, mean, rstd = sg.layer_norm(x, w, b, stats=True, out=at_any(x, offset))
    check(x, w, b, 1e-5, (y, mean, rstd))
    inside = at_any(x, offset)
    got = sg.layer_norm(inside, w, b, stats=True, out=inside)
    assert got[0] is inside and all(torch.equal(p, q) for p, q in zip(got, (y, mean, rstd)))
    want = sg.layer_norm_backward(dy, x, mean, rstd, w, out=at_any(x, offset))
    for which in range(2):
        inside = at_any((dy, x)[which], offset)
        got = sg.layer_norm_backward(*((inside, x), (dy, inside))[which], mean, rstd, w, out=inside)
        assert got[0] is inside and all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("params", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_parameters_at_any_alignment(cols, dtype, params):
    """Each type of weight and bias in each layout, and vectors that begin one element after a 16-byte boundary."""
    x, w, b, dy = problem(200, cols, dtype, params=params)
    got = sg.layer_norm(x, w, b, stats=True)
    check(x, w, b, 1e-5, got)
    grads = sg.layer_norm_backward(dy, x, *got[1:], w)
    same = sg.layer_norm_backward(dy, x, *got[1:], w.float())
    assert all(torch.equal(p, q) for p, q in zip(grads, same))
    w1, b1 = (torch.zeros(cols + 1, dtype=params, device="cuda")[1:].copy_(t) for t in (w, b))
    assert w1.data_ptr() % 16 != 0
    for pw, pb in ((w1, b1), (w, b1), (w1, b)):
        assert all(torch.equal(p, q) for p, q in zip(sg.layer_norm(x, pw, pb, stats=True), got))
    assert all(torch.equal(p, q) for p, q in zip(sg.layer_norm_backward(dy, x, *got[1:], w1), grads))


def test_sums_at_any_alignment():
    """mean, rstd, dweight and dbias that begin anywhere."""
    x, w, b, dy = problem(300, 1000, torch.bfloat16)
    _, mean, rstd = sg.layer_norm(x, w, b, stats=True)
    want = sg.layer_norm_backward(dy, x, mean, rstd, w)
    m1, r1 = (torch.zeros(301, device="cuda")[1:].copy_(t) for t in (mean, rstd))
    held = torch.full((2004,), float("nan"), device="cuda")
    got = sg.layer_norm_backward(dy, x, m1, r1, w, dweight=held[1:1001], dbias=held[1002:2002])
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert torch.isnan(held[[0, 1001, 2002, 2003]]).all()
