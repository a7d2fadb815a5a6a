"""GPU tests of layer norm on rows whose mean is large beside their spread, against plain 64-bit forms.

Bounds, with u = 2^-24, STEPS = 64 as in test_gpu_layer_norm, M the mean and s the spread, the root of the variance.
The first mean m of a row is off by at most em = STEPS u mean|x|. Where |m| is above 4 s the mean of the distances
from it corrects it, which is off by STEPS u mean|x - m| (the distances' own roundings among it), and mean|x - m| by
em at most from mean|x - M|; elsewhere em itself is at most STEPS u (mean|x - M| + |M|). So both ways what y takes
for the mean is off by at most e2 = STEPS u (mean|x - M| + em + 4.1 s).
  mean   by u |M| more
  rstd   the squares' sum is off by STEPS u, two roundings more on the way; a mean that is off by e2 adds 2 e2 / s +
         (e2 / s)^2, s with eps. rstd is off by half of that; `rel` below is the whole.
  y      |w| (|x - M| rstd (rel + 4 u) + (e2 + 2 u em) rstd) + u |y|, and one rounding to its type
Constant rows have distances that are few units in the last place of x, all the same, whose sums are exact: the
corrected mean is the number itself and the variance 0.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

from test_gpu_layer_norm import STEPS, TYPES, U, plain, rand, rounding

# a size or two of each layout of a row
COLS = [7, 64, 250, 500, 777, 1000, 1024, 2000, 4000, 4096, 5000, 8000, 12287, 12288, 15000, 16384, 16385, 20000]


def check(x, w, b, eps, got):
    y, mean, rstd = got
    w = torch.ones(x.shape[1], device="cuda") if w is None else w
    b = torch.zeros(x.shape[1], device="cuda") if b is None else b
    Y, M, R = plain(x, w, b, eps)
    d = (x.double() - M).abs()
    em = STEPS * U * x.double().abs().mean(1, keepdim=True)
    spread = d.square().mean(1, keepdim=True)
    e2 = STEPS * U * (d.mean(1, keepdim=True) + em + 4.1 * spread.sqrt())
    s = (spread + eps).sqrt()
    rel = STEPS * U + 2 * e2 / s + (e2 / s).square() + 4 * U
    assert ((mean.double()[:, None] - M).abs() <= e2 + U * M.abs()).all()
    assert ((rstd.double()[:, None] - R).abs() <= rel * R).all()
    tol = w.double().abs() * R * (d * (rel + 4 * U) + e2 + 2 * U * em) + U * Y.abs()
    assert ((y.double() - Y).abs() <= tol + rounding(Y.abs() + tol, x.dtype)).all()


def at_any(x, offset):
    """x in rows that begin `offset` elements after a 16-byte boundary."""
    pitch = (x.shape[1] + offset + 7) // 8 * 8
    return torch.zeros(x.shape[0], pitch, dtype=x.dtype, device="cuda")[:, offset:offset + x.shape[1]].copy_(x)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_constant_rows(cols, dtype, offset):
    values = torch.tensor([0.1, -0.7, 3.3, 1000.1, 10000.1, 2.0 ** -10 + 2.0 ** -33, 1.0 - 2.0 ** -24]).to(dtype)
    x = at_any(values[:, None].expand(-1, cols), offset)
    w, b = (1 + 0.3 * rand(cols, seed=1)).cuda(), rand(cols, seed=2).cuda()
    y, mean, rstd = sg.layer_norm(x, w, b, stats=True)
    assert torch.equal(mean, values.float().cuda())
    assert torch.equal(y, b.to(dtype).expand_as(y))
    assert torch.equal(rstd, torch.full_like(rstd, 1e-5 ** -0.5)) or (rstd * 1e-5 ** 0.5 - 1).abs().max() <= 4 * U
    y, mean, rstd = sg.layer_norm(x, eps=0.0, stats=True)
    assert torch.equal(mean, values.float().cuda()) and (rstd == float("inf")).all() and torch.isnan(y).all()


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_mean_far_from_zero(cols, dtype, offset):
    """Spreads from the mean's own size to its last bits."""
    far = torch.tensor([1.0, 30.0, 1000.1, -10000.1, 0.1])
    x = at_any(torch.cat([far[:, None] * (1 + spread * rand(5, cols, seed=cols)) for spread in (1.0, 1e-2, 1e-4, 1e-6, 2e-7)])
               .to(dtype), offset)
    w, b = (1 + 0.3 * rand(cols, seed=1)).cuda(), rand(cols, seed=2).cuda()
    for eps in (1e-5, 1e-12):
        check(x, w, b, eps, sg.layer_norm(x, w, b, eps=eps, stats=True))


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("cols", COLS)
def test_one_element_differs(cols, offset):
    """Rows of one value but for one element, from the value's last bit on."""
    x = torch.tensor([0.1, 3.3, 1000.1, -10000.1])[:, None].repeat(6, cols)
    for r in range(x.shape[0]):
        x[r, (r * 31) % cols] *= 1 + 2.0 ** (-22 + 2 * (r // 4))
    x = at_any(x, offset)
    check(x, None, None, 0.0, sg.layer_norm(x, eps=0.0, stats=True))


@pytest.mark.parametrize("cols", [64, 250, 512, 1024, 4096])
def test_rows_do_not_change_their_neighbours(cols):
    """Rows whose squares are taken again lie among others: each row has the bits that it has with its like, and so
    has each of many rows that a block takes in turn. (With its like at the same pitch: one row alone counts as
    aligned.)"""
    kinds = torch.stack([rand(cols, seed=1), 0.1 + torch.zeros(cols), 1000.1 * (1 + 2e-7 * rand(cols, seed=2)),
                         5 + rand(cols, seed=3)])
    x = kinds[torch.randint(4, (6000,), generator=torch.Generator().manual_seed(5))].cuda()
    got = sg.layer_norm(x, stats=True)
    for row in kinds.cuda():
        alone = [t[0] for t in sg.layer_norm(row[None].repeat(2, 1), stats=True)]
        same = (x == row).all(1)
        assert same.sum() > 1000
        for a, g in zip(alone, got):
            assert (g[same] == a).all()
