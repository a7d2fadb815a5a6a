"""GPU test of examples/f8_linear_layer.py: its products and update against the plain forms in 64
bits, and that it learns.

Bounds. An e4m3 number is within 2^-4 of its value relative to it, or within 2^-10 of the block's
scale where that is more; the scale is the block's largest number over 448, so that second error is
at most t = 2^-10 / 448 of the largest. A product of two quantised matrices A, B is therefore within
    (2^-4 |A| + t max|A|) |B| + |A| (2^-4 |B| + t max|B|) + (the same errors multiplied)
of the exact one; the tests take 1.1 times the first two, and the rounding to the result's type.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "f8_linear_layer", os.path.join(ROOT, "examples", "f8_linear_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def bound(a, b, rounding):
    """Of a @ b (64 bits) from 8-bit copies of both."""
    a, b = a.abs(), b.abs()
    ea = 2.0 ** -4 * a + 2.0 ** -10 / 448 * a.max()
    eb = 2.0 ** -4 * b + 2.0 ** -10 / 448 * b.max()
    return 1.1 * (ea @ b + a @ eb) + rounding * (a @ b)


@pytest.mark.parametrize("tokens,inputs,outputs", [(1, 64, 48), (130, 200, 129), (300, 129, 257)])
def test_products(example, tokens, inputs, outputs):
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, inputs, generator=g).bfloat16()
    dy = torch.randn(tokens, outputs, generator=g).bfloat16()
    w = torch.randn(outputs, inputs, generator=g)
    layer = example.Linear8(w.cuda())
    y = layer.forward(x.cuda())
    dx = layer.backward(dy.cuda())
    x, dy, w = x.double(), dy.double(), w.double()
    for got, a, b, rounding in ((y, x, w.t(), 2.0 ** -7), (dx, dy, w, 2.0 ** -7),
                                (layer.grad, dy.t(), x, 2.0 ** -20)):
        assert ((got.cpu().double() - a @ b).abs() <= bound(a, b, rounding)).all()
    once = layer.grad.clone()
    layer.forward(x.bfloat16().cuda())
    layer.backward(dy.bfloat16().cuda())
    assert torch.equal(layer.grad, 2 * once)  # the same batch again is added


def test_update(example):
    """Against the plain steps in 64 bits; the bound is test_gpu_orthogonalize's."""
    g = torch.Generator().manual_seed(3)
    w, m, grad = (torch.randn(96, 160, generator=g) for _ in range(3))
    layer = example.Linear8(w.cuda())
    layer.momentum.copy_(m)
    layer.grad.copy_(grad)
    layer.update(0.05, momentum=0.5, decay=0.1)
    x = (torch.tensor(0.5) * m + grad).double()
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        s = x @ x.t()
        x = 3.4445 * x + (-4.7750 * s + 2.0315 * (s @ s)) @ x
    want = (1 - 0.05 * 0.1) * w.double() - 0.05 * x
    tol = 0.05 * (2.0 ** -20 * sum(4.0 ** k for k in range(5)) + 2.0 ** -22) * x.norm() \
        + 2.0 ** -22 * want.norm()
    assert (layer.weight.cpu().double() - want).norm() <= tol
    assert layer.batches == 0


def test_learns_and_serves(example):
    x, target, w1, w2 = example.problem(512, 128, seed=1)
    model = example.Pair(w1, w2)
    losses = example.train(model, x, target, steps=20, rate=0.05)
    assert losses[-1] < 0.5 * losses[0]
    one, all_ = model.serve(x[:1]), model.serve(x)
    # the same 8-bit numbers, added in another order: FP32 sums rounded to BF16, twice
    assert (one - all_[:1]).abs().max() <= 2.0 ** -4 * all_[:1].abs().max()
