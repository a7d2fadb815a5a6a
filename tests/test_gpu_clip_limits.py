"""GPU tests of the limits of clipping: which numbers max_norm and eps may be, to the last bit of the factor.

Gradients are whole numbers, whose squares and their sum are exact, so that the norm is the 64-bit root that the host
computes too (both are rounded correctly), and the factor the 64-bit quotient rounded once to FP32. A clipped FP32
gradient is then one FP32 product, bit for bit.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg


def problem():
    g = torch.Generator().manual_seed(7)
    return [torch.randint(-9, 10, (n,), generator=g).float().cuda() for n in (1, 77, 40000, 5)]


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-3, 0.1])
@pytest.mark.parametrize("limit", [0.1, 0.3e-3 * math.sqrt(77777), 1 / 3, 1e-6, 7.3e-5, 100.1, 0.5, 1e-30])
def test_limits_that_fp32_does_not_hold(limit, eps):
    grads = problem()
    norm = math.sqrt(sum(g.double().square().sum().item() for g in grads))
    factor = torch.tensor(limit / (norm + eps), dtype=torch.float64).float().cuda()
    out = [torch.empty_like(g) for g in grads]
    got = sg.clip_grad_norm(grads, limit, eps=eps, out=out)
    assert got.item() == torch.tensor(norm, dtype=torch.float64).float().item()
    assert all(torch.equal(o, g * factor) for o, g in zip(out, grads))
    want = [o.clone() for o in out]
    sg.clip_grad_norm(grads, limit, eps=eps)
    assert all(torch.equal(g, w) for g, w in zip(grads, want))


def test_a_limit_just_above_the_norm_changes_nothing():
    """FP32 would round this one to the norm, and eps would put the factor below 1."""
    grads = problem()
    before = [g.clone() for g in grads]
    norm = math.sqrt(sum(g.double().square().sum().item() for g in grads))
    sg.clip_grad_norm(grads, norm * (1 + 1e-12) + 1e-9, eps=1e-9)
    assert all(torch.equal(g, b) for g, b in zip(grads, before))


@pytest.mark.parametrize("limit", [2.0 ** -20, 2.0 ** -100, 3e-44, 1e-60, 1e-70, 1e-300])
@pytest.mark.parametrize("power", [0, 60, 100, 126])
def test_factors_below_fp32(limit, power):
    """Large gradients and small limits, whose factor is no FP32 number although results are: off by the factor's,
    the norm's and the product's roundings (40 u, as in test_gpu_clip), or a smallest step."""
    g = (1 + torch.rand(5000, generator=torch.Generator().manual_seed(1))).cuda() * 2.0 ** power
    g[1::2] *= 2.0 ** -24
    norm = g.double().square().sum().sqrt().item()
    out = [torch.empty_like(g)]
    sg.clip_grad_norm([g], limit, eps=0.0, out=out)
    want = g.double() * (limit / norm)
    assert ((out[0].double() - want).abs() <= 40 * 2.0 ** -24 * want + 2.0 ** -149).all()
