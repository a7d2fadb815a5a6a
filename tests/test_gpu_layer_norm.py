"""GPU tests of layer norm and its gradients against plain 64-bit forms and against differences.

Bounds, with u = 2^-24, half a step of FP32, and STEPS = 64: a sum along a row passes through at most
16 + 5 + 32 additions (a thread's elements, a warp's lanes, the warps) and a few other roundings.
  mean   off by em = STEPS u mean|x|
  rstd   the variance is off by STEPS u and by 2 em / s + (em / s)^2 relative to itself (s its root),
         rstd by half as much and 2 u; `rel` below is twice that
  y      |w| (|x - mean| rstd (rel + 4 u) + em rstd) + u |y|, and one rounding to its type
  dx     with h and g off by 2 u each: rstd (8 u (|g| + |s1| + |h s2|) + STEPS u (mean|g| + |h| mean|g h|)),
         and one rounding
  dw     up to 500 additions of a thread's rows, 17 more in its block and 15 of parts in FP32:
         (min(rows, 512) + 24) u sum |dy h|; db alike
In rows that are read more than once sums are more exact than that. A rounding to a type t is off by at
most finfo(t).eps / 2 of the value and, in FP16, by half its smallest step, 2^-25.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

U, STEPS = 2.0 ** -24, 64
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# around every limit between the layouts of a row, and past the rows that stay in registers
SHAPES = [(1, 1), (1, 7), (3, 64), (40, 65), (5, 256), (300, 257), (7, 512), (33, 777), (9, 1024),
          (4, 1025), (5, 2048), (3, 2056), (1, 4096), (3, 4096), (3, 4100), (2, 8192), (3, 8200), (2, 16384),
          (2, 16392), (1, 40001)]


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def rounding(t, dtype):
    return torch.finfo(dtype).eps / 2 * t.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def plain(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()
    return (x - mean) * rstd * w.double() + b.double(), mean, rstd


def check(x, w, b, eps, got):
    y, mean, rstd = got
    assert y.dtype == x.dtype and y.shape == x.shape
    assert mean.dtype == rstd.dtype == torch.float32 and mean.shape == rstd.shape == x.shape[:1]
    w = torch.ones(x.shape[1], device="cuda") if w is None else w
    b = torch.zeros(x.shape[1], device="cuda") if b is None else b
    Y, M, R = plain(x, w, b, eps)
    d = x.double() - M
    em = STEPS * U * x.double().abs().mean(1, keepdim=True)
    s = (d.square().mean(1, keepdim=True) + eps).sqrt()
    rel = STEPS * U + 2 * em / s + (em / s).square() + 2 * U
    assert ((mean.double()[:, None] - M).abs() <= em + U * M.abs()).all()
    assert ((rstd.double()[:, None] - R).abs() <= rel * R).all()
    tol = w.double().abs() * (d.abs() * R * (rel + 4 * U) + em * R) + U * Y.abs() + rounding(Y, x.dtype)
    assert ((y.double() - Y).abs() <= tol).all()


def plain_backward(dy, x, mean, rstd, w):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    h, g = (x - mean) * rstd, dy * w.double()
    s1, s2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    return rstd * (g - s1 - h * s2), (dy * h).sum(0), dy.sum(0), (h, g, s1, s2, rstd, dy)


def check_backward(dy, x, mean, rstd, w, got, beta=0.0, before=(0.0, 0.0)):
    dx, dw, db = got
    w = torch.ones(x.shape[1], device="cuda") if w is None else w
    DX, DW, DB, (h, g, s1, s2, r, d) = plain_backward(dy, x, mean, rstd, w)
    assert dx.dtype == x.dtype and dw.dtype == db.dtype == torch.float32
    tol = r * (8 * U * (g.abs() + s1.abs() + (h * s2).abs())
               + STEPS * U * (g.abs().mean(1, keepdim=True) + h.abs() * (g * h).abs().mean(1, keepdim=True)))
    assert ((dx.double() - DX).abs() <= tol + rounding(DX, x.dtype)).all()
    steps = (min(x.shape[0], 512) + 24) * U
    for got_, want, terms, old in ((dw, DW, (d * h).abs().sum(0), before[0]), (db, DB, d.abs().sum(0), before[1])):
        want = want + beta * old
        assert ((got_.double() - want).abs() <= steps * terms + 2 * U * want.abs()).all()


def problem(rows, cols, dtype, seed=0, params=torch.float32):
    x = (rand(rows, cols, seed=seed) * torch.exp(rand(rows, 1, seed=seed + 1)) + rand(rows, 1, seed=seed + 2))
    w, b = 1 + 0.3 * rand(cols, seed=seed + 3), 0.3 * rand(cols, seed=seed + 4)
    dy = rand(rows, cols, seed=seed + 5)
    return [t.cuda() for t in (x.to(dtype), w.to(params), b.to(params), dy.to(dtype))]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype):
    x, w, b, dy = problem(*shape, dtype)
    got = sg.layer_norm(x, w, b, stats=True)
    check(x, w, b, 1e-5, got)
    assert torch.equal(sg.layer_norm(x, w, b), got[0])
    check_backward(dy, x, *got[1:], w, sg.layer_norm_backward(dy, x, *got[1:], w))


@pytest.mark.parametrize("params", TYPES)
@pytest.mark.parametrize("shape", [(20, 300), (3, 9000), (2, 20000)], ids=lambda s: "x".join(map(str, s)))
def test_parameters(shape, params):
    """Each type of weight and bias, one of them, and none."""
    x, w, b, dy = problem(*shape, torch.bfloat16, params=params)
    for pw, pb in ((w, b), (w, None), (None, b), (None, None)):
        got = sg.layer_norm(x, pw, pb, eps=1e-3, stats=True)
        check(x, pw, pb, 1e-3, got)
    mean, rstd = got[1:]
    check_backward(dy, x, mean, rstd, w, sg.layer_norm_backward(dy, x, mean, rstd, w))
    dx, dw, db = sg.layer_norm_backward(dy, x, mean, rstd)
    assert dw is None and db is None
    full = sg.layer_norm_backward(dy, x, mean, rstd, torch.ones_like(w))
    assert torch.equal(dx, full[0])
    into = [torch.empty(shape[1], device="cuda") for _ in range(2)]
    alone = sg.layer_norm_backward(dy, x, mean, rstd, dweight=into[0], dbias=into[1])
    assert all(torch.equal(p, q) for p, q in zip(alone, full)) and alone[1] is into[0]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(5000, 300), (3000, 700), (2500, 1501), (700, 4095), (310, 4608), (310, 6144),
                                   (310, 6145), (310, 8193), (310, 10240), (310, 12288), (310, 12289), (310, 12296),
                                   (160, 16384)], ids=lambda s: "x".join(map(str, s)))
def test_layouts_of_long_rows(shape, dtype, offset):
    """Several rows for each block in the layouts of long rows and of unaligned ones."""
    x, w, b, dy = problem(*shape, dtype)
    pitch = (shape[1] + offset + 7) // 8 * 8 + offset
    x, dy = (torch.cat((t, t.new_zeros(shape[0], pitch - shape[1])), 1)[:, :shape[1]] for t in (x, dy))
    got = sg.layer_norm(x, w, b, stats=True)
    check(x, w, b, 1e-5, got)
    check_backward(dy, x, *got[1:], w, sg.layer_norm_backward(dy, x, *got[1:], w))
    alone, *none = sg.layer_norm_backward(dy, x, *got[1:])
    assert none == [None, None]
    check_backward(dy, x, *got[1:], None, (alone, *sg.layer_norm_backward(dy, x, *got[1:], torch.ones_like(w))[1:]))


@pytest.mark.parametrize("shape", [(5000, 40), (3000, 130), (2500, 512), (2000, 1500), (700, 4096),
                                   (400, 8192), (70000, 16), (60, 20000)], ids=lambda s: "x".join(map(str, s)))
def test_many_rows(shape):
    """Several rows for each block."""
    x, w, b, dy = problem(*shape, torch.bfloat16)
    got = sg.layer_norm(x, w, b, stats=True)
    check(x, w, b, 1e-5, got)
    check_backward(dy, x, *got[1:], w, sg.layer_norm_backward(dy, x, *got[1:], w))


def test_more_rows_than_one_sum_holds():
    """More than 512 rows for each of the blocks that fill the GPU."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(5500000, 8, generator=g, device="cuda").half() for _ in range(2))
    w, b = 1 + 0.3 * rand(8, seed=2).cuda(), rand(8, seed=3).cuda()
    got = sg.layer_norm(x, w, b, stats=True)
    check(x, w, b, 1e-5, got)
    check_backward(dy, x, *got[1:], w, sg.layer_norm_backward(dy, x, *got[1:], w))


@pytest.mark.parametrize("cols", [33, 390, 4000, 8192, 17000])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned(cols, offset, dtype):
    """Views into larger matrices, whose other elements are left alone."""
    def view(t):
        buf = torch.full((9, cols + 11), float("nan"), dtype=dtype, device="cuda")
        v = buf[2:7, offset:offset + cols]
        v.copy_(t)
        return buf, v

    x, w, b, dy = problem(5, cols, dtype)
    (_, xv), (_, dyv), (ybuf, yv) = view(x), view(dy), view(torch.zeros_like(x))
    y, mean, rstd = sg.layer_norm(xv, w, b, stats=True, out=yv)
    assert y is yv
    check(x, w, b, 1e-5, (y, mean, rstd))
    yv.fill_(float("nan"))
    assert torch.isnan(ybuf).all()
    dbuf, dxv = view(torch.zeros_like(x))
    got = sg.layer_norm_backward(dyv, xv, mean, rstd, w, out=dxv)
    assert got[0] is dxv
    check_backward(dy, x, mean, rstd, w, got)
    dxv.fill_(float("nan"))
    assert torch.isnan(dbuf).all()


@pytest.mark.parametrize("cols", [100, 3000, 16400])
def test_in_place_and_added_up(cols):
    x, w, b, dy = problem(700, cols, torch.bfloat16)
    want = sg.layer_norm(x, w, b, stats=True)
    y = x.clone()
    got = sg.layer_norm(y, w, b, stats=True, out=y)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    mean, rstd = want[1:]
    first = sg.layer_norm_backward(dy, x, mean, rstd, w)
    for buf in (dy.clone(), x.clone()):
        a, c = (buf, x) if torch.equal(buf, dy) else (dy, buf)
        again = sg.layer_norm_backward(a, c, mean, rstd, w, out=buf)
        assert again[0] is buf and all(torch.equal(p, q) for p, q in zip(again, first))
    dw, db = first[1].clone(), first[2].clone()
    got = sg.layer_norm_backward(dy, x, mean, rstd, w, dweight=dw, dbias=db, beta=0.5)
    assert got[1] is dw and got[2] is db
    check_backward(dy, x, mean, rstd, w, got, 0.5, (first[1].double(), first[2].double()))
    nan = [torch.full((cols,), float("nan"), device="cuda") for _ in range(2)]
    got = sg.layer_norm_backward(dy, x, mean, rstd, w, dweight=nan[0], dbias=nan[1])
    assert all(torch.equal(p, q) for p, q in zip(got, first))  # beta = 0 does not read them


@pytest.mark.parametrize("cols", [37, 600])
def test_gradients_are_those_of_differences(cols):
    """Against central differences of the 64-bit form: with a step of 1e-4 they are off by about 1e-8
    (the third derivative is of the order of one) and by 1e-15 / 1e-4; FP32's part is under 1e-5."""
    x, w, b, dy = problem(3, cols, torch.float32, seed=9)
    _, mean, rstd = sg.layer_norm(x, w, b, stats=True)
    dx, dw, db = sg.layer_norm_backward(dy, x, mean, rstd, w)
    step = 1e-4

    def loss(x, w, b):
        return (plain(x, w, b, 1e-5)[0] * dy.double()).sum().item()

    for t, grad in ((x, dx), (w, dw), (b, db)):
        for i in range(0, t.numel(), max(1, t.numel() // 20)):
            ends = []
            for sign in (1, -1):
                moved = [u.double().clone() for u in (x, w, b)]
                moved[0 if t is x else 1 if t is w else 2].view(-1)[i] += sign * step
                ends.append(loss(*moved))
            want = (ends[0] - ends[1]) / (2 * step)
            assert abs(grad.view(-1)[i].item() - want) <= 1e-5 * (1 + grad.abs().max().item())


@pytest.mark.parametrize("cols", [64, 1000, 4096, 20000])
def test_mean_far_from_zero(cols):
    """The variance is that of the distances, not a difference of squares."""
    x = (1000 + rand(4, cols, seed=1)).cuda()
    got = sg.layer_norm(x, stats=True)
    check(x, None, None, 1e-5, got)
    # s is about 1, and the distances themselves are good to one step of 1000
    assert (got[0].double().square().mean(1) - 1).abs().max() <= 1e-3


@pytest.mark.parametrize("cols", [48, 4096, 17000])
def test_not_finite_stays_in_its_row(cols):
    x, w, b, dy = problem(6, cols, torch.float32)
    want = sg.layer_norm(x, w, b, stats=True)
    grads = sg.layer_norm_backward(dy, x, *want[1:], w)
    bad = x.clone()
    bad[1, 3], bad[4, cols - 1] = float("nan"), float("inf")
    got = sg.layer_norm(bad, w, b, stats=True)
    back = sg.layer_norm_backward(dy, bad, *got[1:], w)
    for r in range(6):
        if r in (1, 4):
            assert torch.isnan(got[0][r]).all() and torch.isnan(back[0][r]).all()
        else:
            assert torch.equal(got[0][r], want[0][r]) and torch.equal(back[0][r], grads[0][r])
    assert torch.isnan(back[1]).all() and torch.equal(back[2], grads[2])


def test_constant_rows_and_magnitudes():
    x = torch.full((2, 300), 7.0).cuda()
    assert (sg.layer_norm(x) == 0).all()
    for scale in (2.0 ** -60, 2.0 ** 40):
        x = (rand(3, 500, seed=2) * scale).cuda()
        check(x, None, None, 0.0, sg.layer_norm(x, eps=0.0, stats=True))


@pytest.mark.parametrize("cols", [1, 300, 5000, 20000])
def test_constant_rows_without_eps(cols):
    # variance 0 and eps 0: 1 / sqrt(0)
    x = torch.full((2, cols), 3.0).cuda()
    y, mean, rstd = sg.layer_norm(x, eps=0.0, stats=True)
    assert (mean == 3).all() and (rstd == float("inf")).all() and torch.isnan(y).all()


def test_no_rows():
    x = torch.empty(0, 50, device="cuda")
    y, mean, rstd = sg.layer_norm(x, stats=True)
    assert y.shape == (0, 50) and mean.shape == (0,)
    w, dw, db = torch.ones(50, device="cuda"), torch.ones(50, device="cuda"), torch.ones(50, device="cuda")
    dx, *got = sg.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 50) and all((t == 0).all() for t in got)
    sg.layer_norm_backward(x, x, mean, rstd, w, dweight=dw, dbias=db, beta=2.0)
    assert (dw == 2).all() and (db == 2).all()


@pytest.mark.parametrize("shape", [(3000, 512), (500, 4096), (64, 9000)], ids=lambda s: "x".join(map(str, s)))
def test_same_bits_every_time(shape):
    x, w, b, dy = problem(*shape, torch.bfloat16)
    first = sg.layer_norm(x, w, b, stats=True)
    back = sg.layer_norm_backward(dy, x, *first[1:], w)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(sg.layer_norm(x, w, b, stats=True), first))
        again = sg.layer_norm_backward(dy, x, *first[1:], w)
        assert all(torch.equal(p, q) for p, q in zip(again, back))


def test_offsets_past_32_bits():
    rows, cols = 1 << 20, 4160
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = rand(3, cols, seed=1).to(torch.bfloat16).cuda()
    x[:, ::2] = 1.0
    x[-3:] = tail
    y, mean, rstd = sg.layer_norm(x, stats=True)
    check(tail, None, None, 1e-5, (y[-3:], mean[-3:], rstd[-3:]))
    dy = y  # (any values)
    want = sg.layer_norm_backward(dy[-3:], x[-3:], mean[-3:], rstd[-3:])[0].clone()
    dx, _, _ = sg.layer_norm_backward(dy, x, mean, rstd, out=y)
    assert torch.equal(dx[-3:], want)


def test_another_stream_and_a_graph():
    x, w, b, dy = problem(300, 1000, torch.bfloat16)

    def chain():
        y, mean, rstd = sg.layer_norm(x, w, b, stats=True)
        return (y, *sg.layer_norm_backward(dy, x, mean, rstd, w))

    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    dy.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
    assert all(torch.equal(p.float(), 2 * q.float()) for p, q in zip(got[1:], want[1:]))


def test_refusals_on_the_gpu():
    x, w = torch.zeros(4, 8, device="cuda"), torch.ones(8, device="cuda")
    s = torch.ones(4, device="cuda")
    for bad in (w[:7], torch.ones(16, device="cuda")[::2], torch.ones(8, 1, device="cuda")):
        with pytest.raises(ValueError):
            sg.layer_norm(x, bad)
        with pytest.raises(ValueError):
            sg.layer_norm_backward(x, x, s, s, bad)
    with pytest.raises(TypeError):
        sg.layer_norm(x, w.double())
    with pytest.raises(TypeError):  # two types of parameters
        sg.layer_norm(x, w, w.half())
    with pytest.raises(ValueError):  # a parameter on the CPU
        sg.layer_norm(x, w.cpu())
    with pytest.raises(ValueError):
        sg.layer_norm(x[:, :0])
    with pytest.raises(ValueError, match="overlap"):
        sg.layer_norm(x[:1].expand(4, 8))
    with pytest.raises(ValueError):
        sg.layer_norm(x.t())
    with pytest.raises(TypeError):  # the result's type
        sg.layer_norm(x, out=x.half())
    with pytest.raises(ValueError):
        sg.layer_norm(x, out=torch.zeros(4, 9, device="cuda"))
    with pytest.raises(TypeError):
        sg.layer_norm_backward(x.half(), x, s, s)
    with pytest.raises(ValueError):
        sg.layer_norm_backward(x, x, s[:3], s)
    with pytest.raises(TypeError):
        sg.layer_norm_backward(x, x, s.double(), s)
    with pytest.raises(ValueError):  # nothing to scale
        sg.layer_norm_backward(x, x, s, s, w, beta=1.0)
    with pytest.raises(ValueError):  # one buffer for both sums
        sg.layer_norm_backward(x, x, s, s, w, dweight=w, dbias=w)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(sg.SgemmError) as e:
            sg.layer_norm(x, eps=eps)
        assert e.value.status == -9
