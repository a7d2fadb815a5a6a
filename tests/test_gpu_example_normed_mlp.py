"""GPU test of examples/normed_mlp.py: layer norm, the 8-bit products, clipping, the update and the layers
in 8-bit integers run together, each stage against its 64-bit form on what the stage before it left.

Bounds. Stages are those of their own tests. The served block is compared with the 64-bit block on the
integers' values: a row's quantisation is within half a step of its scale, s / 2 per element, so that a
product of quantised rows is off by at most (s_x / 2) sum |w| + (s_w / 2) sum |x| + k s_x s_w / 4; the
results' types add half a step each (2^-9 relative for BF16).
"""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HALF = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def example():
    path = os.path.join(ROOT, "examples")
    sys.path.insert(0, path)
    try:
        spec = importlib.util.spec_from_file_location("normed_mlp", os.path.join(path, "normed_mlp.py"))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    finally:
        sys.path.remove(path)
    return mod


def block_of(example, tokens, width, seed):
    x, target, w1, w2 = example.problem(tokens, width, seed=seed)
    block = example.Block(w1, w2)
    g = torch.Generator().manual_seed(seed + 7)
    block.weight.copy_(1 + 0.2 * torch.randn(width, generator=g))
    block.bias.copy_(0.2 * torch.randn(width, generator=g))
    return block, x, target


def normed(x, weight, bias):
    x = x.double()
    d = x - x.mean(1, keepdim=True)
    return d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * weight.double() + bias.double()


@pytest.mark.parametrize("tokens,width", [(1, 64), (150, 200), (300, 136)])
def test_a_step_stage_by_stage(example, tokens, width):
    block, x, _ = block_of(example, tokens, width, tokens)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(tokens, width, generator=g).bfloat16().cuda()
    y = block.forward(x)
    h = example.sg.layer_norm(x, block.weight, block.bias)
    want = normed(x, block.weight, block.bias)
    assert ((h.double() - want).abs() <= HALF * want.abs() + 2.0 ** -16 * (1 + want.abs())).all()
    assert torch.equal(y, x + block.second.forward(block.a))
    dx = block.backward(dy)
    # the gradients of the norm, from the gradient of its result
    r = block.rstd.double()[:, None]
    hat = (x.double() - block.mean.double()[:, None]) * r
    d = block.dh.double() * block.weight.double()
    core = r * (d - d.mean(1, keepdim=True) - hat * (d * hat).mean(1, keepdim=True))
    size = r * (d.abs() + d.abs().mean(1, keepdim=True) + hat.abs() * (d * hat).abs().mean(1, keepdim=True))
    # (rounded to BF16, added to dy, rounded again)
    assert ((dx.double() - (core + dy.double())).abs()
            <= 2.0 ** -16 * size + HALF * core.abs() + 1.01 * HALF * (core + dy.double()).abs()).all()
    for got, terms in ((block.dweight, block.dh.double() * hat), (block.dbias, block.dh.double())):
        assert ((got.double() - terms.sum(0)).abs() <= 2.0 ** -14 * terms.abs().sum(0)).all()
    # a second batch is added
    once = [t.clone() for t in (block.dweight, block.dbias, block.first.grad, block.second.grad)]
    block.forward(x)
    block.backward(dy)
    for t, o in zip((block.dweight, block.dbias, block.first.grad, block.second.grad), once):
        assert (t - 2 * o).abs().max() <= 2.0 ** -22 * o.abs().max()


def test_update_clips_what_it_applies(example):
    block, x, target = block_of(example, 200, 128, 3)
    block.forward(x)
    block.backward(torch.randn(200, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda())
    grads = [t.double() for t in (block.first.grad, block.second.grad, block.dweight, block.dbias)]
    weight, bias = block.weight.double(), block.bias.double()
    norm = sum(g.square().sum() for g in grads).sqrt().item()
    got = block.update(0.1, 0.25 * norm)
    assert got.item() == pytest.approx(norm, rel=2.0 ** -18)
    factor = 0.25 * norm / (norm + 1e-6)
    for new, old, g in ((block.weight, weight, grads[2]), (block.bias, bias, grads[3])):
        want = old - 0.1 * factor * g
        assert ((new.double() - want).abs() <= 2.0 ** -20 * (want.abs() + (0.1 * g).abs())).all()
    assert block.batches == 0 and block.first.batches == 0


@pytest.mark.parametrize("tokens,width", [(1, 128), (5, 200), (40, 136), (300, 256)])
def test_serving(example, tokens, width):
    block, x, _ = block_of(example, tokens, width, 11)
    serve = block.quantize()
    y = serve(x)
    assert y.dtype == x.dtype and y.data_ptr() != x.data_ptr()

    def product(t, w, extra):
        """t w^T and how far the integers may be off, t itself being off by `extra`."""
        t, w = t.double(), w.double()
        st, sw = (t.abs() + extra).amax(1, keepdim=True) / 127, w.abs().amax(1, keepdim=True) / 127
        et, ew = st / 2 + extra, sw / 2
        return t @ w.t(), 1.001 * (et @ w.abs().t() + t.abs() @ ew.expand_as(w).t() + et @ ew.expand_as(w).t())

    h = normed(x, block.weight, block.bias)
    z, ez = product(h, block.first.weight, HALF * h.abs() + 2.0 ** -16 * (1 + h.abs()))
    ez = ez + HALF * (z.abs() + ez)
    a = z.clamp_min(0)
    out, eo = product(a, block.second.weight, ez)
    out = out + x.double()
    assert ((y.double() - out).abs() <= eo + HALF * (out.abs() + eo)).all()
    # a token alone is the same token (whole numbers do not depend on the batch)
    assert torch.equal(serve(x[:1]), y[:1])


def test_runs(example):
    block, x, target = block_of(example, 256, 128, 21)
    losses, norms = example.train(block, x, target, steps=3, rate=0.02, limit=0.05)
    assert len(losses) == len(norms) == 3 and all(v == v and v > 0 for v in losses + norms)
