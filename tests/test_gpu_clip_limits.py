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
