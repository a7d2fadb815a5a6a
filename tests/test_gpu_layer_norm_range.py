"""GPU tests of layer norm at both ends of FP32's range, on both sides of the longest row that stays in registers."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

from test_gpu_layer_norm import check, rand

COLS = [48, 300, 777, 1000, 4096, 5000, 8192, 12288, 16384, 16385, 40000]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("far", [0.0, 10.0])
@pytest.mark.parametrize("cols", COLS)
def test_a_variance_beyond_fp32(cols, far, dtype):
    """1 / sqrt of an infinite variance is 0, and y the bias, whatever the row's length."""
    x = (2.0 ** 70 * (far + rand(3, cols, seed=1))).to(dtype).cuda()
    w, b = (1 + 0.3 * rand(cols, seed=2)).cuda(), rand(cols, seed=3).cuda()
    y, mean, rstd = sg.layer_norm(x, w, b, stats=True)
    assert (rstd == 0).all() and torch.equal(y, b.to(dtype).expand_as(y))
    want = x.double().mean(1)
    assert ((mean.double() - want).abs() <= 66 * 2.0 ** -24 * x.double().abs().mean(1)).all()


@pytest.mark.parametrize("cols", COLS)
def test_the_limits_are_held(cols):
    """Spreads from 2^-60 on without eps, magnitudes up to 2^62 / sqrt(cols)."""
    x = rand(3, cols, seed=4).double()
    d = x - x.mean(1, keepdim=True)
    small = x * 2.0 ** -60 / d.square().mean(1, keepdim=True).sqrt() * 1.001  # (a little for the rounding)
    large = x * 2.0 ** 62 / cols ** 0.5 / x.abs().amax(1, keepdim=True) * 0.999
    for t in (small.float().cuda(), large.float().cuda()):
        check(t, None, None, 0.0, sg.layer_norm(t, eps=0.0, stats=True))


def test_the_upper_limit_of_a_very_long_row():
    x = torch.randn(1, 1 << 26, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x *= 2.0 ** 49 * 0.999 / x.abs().max()
    check(x, None, None, 0.0, sg.layer_norm(x, eps=0.0, stats=True))
