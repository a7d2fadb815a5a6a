"""GPU tests of the Newton-Schulz orthogonalisation against the plain iteration in 64 bits.

Bound. One step computed with 22-bit factors and FP32 sums is within EPS = 2^-20 of the exact
step in the Frobenius norm, relative to its result, and a step's map stretches an earlier error by
at most L = max |a + 3 b y + 5 c y^2| over the squares y of the singular values it can meet (4 for
the usual coefficients on [0, 1.2]). So after T steps
    |X - R|_F <= EPS (1 + L + ... + L^(T-1)) |R|_F + u |R|_F
with u = 2^-23, 2^-8, 2^-11 the rounding to out's type. A single FP16 product per factor is 1.2e-3
off on random matrices and 2e-2 on one of low rank with noise, a BF16 one 1e-2 and 0.17: both
outside the 3.3e-4 that five steps have.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

USUAL = (3.4445, -4.7750, 2.0315)
EPS = 2.0 ** -20
ROUND = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def rand(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g)


def plain(g, steps=5, coefficients=USUAL, eps=1e-7):
    a, b, c = coefficients
    x = g.double()
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        if x.shape[-2] <= x.shape[-1]:
            s = x @ x.mT
            x = a * x + (b * s + c * (s @ s)) @ x
        else:
            s = x.mT @ x
            x = a * x + x @ (b * s + c * (s @ s))
    return x


def tolerance(steps, dtype, stretch=4.0):
    return EPS * sum(stretch ** k for k in range(max(steps, 1))) + ROUND[dtype]


def check(got, want, steps, stretch=4.0):
    got = got.cpu()
    w = want.reshape((-1,) + want.shape[-2:])
    g = got.double().reshape(w.shape)
    for i in range(w.shape[0]):
        norm = w[i].norm()
        err = (g[i] - w[i]).norm()
        assert err <= tolerance(steps, got.dtype, stretch) * norm, f"matrix {i}: {err / norm:.3g}"


@pytest.fixture(autouse=True)
def status_clear():
    yield
    assert sg.ns_orthogonalize_status() == (0, 0)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 300), (16, 16), (127, 129), (128, 128), (129, 127),
          (300, 40), (130, 700), (64, 2048), (513, 257), (640, 640)]


@pytest.mark.parametrize("steps", [0, 1, 5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype, steps):
    g = rand(*shape, seed=shape[0]).to(dtype)
    got = sg.orthogonalize(g.cuda(), steps=steps)
    assert got.dtype == dtype and got.shape == g.shape
    check(got, plain(g, steps), steps)


@pytest.mark.parametrize("shape", [(5, 100, 90), (3, 260, 130), (2, 64, 1000), (1, 30, 30)],
                         ids=lambda s: "x".join(map(str, s)))
def test_batch(shape):
    g = rand(*shape, seed=2)
    check(sg.orthogonalize(g.cuda()), plain(g), 5)
    assert torch.equal(sg.orthogonalize(g[0].cuda()), sg.orthogonalize(g.cuda())[0])


@pytest.mark.parametrize("shape", [(256, 512), (700, 300)], ids=lambda s: "x".join(map(str, s)))
def test_weak_directions_survive(shape):
    """Strong directions over weak ones: rounding noise of the strong must not reach the weak."""
    m, n = shape
    g = rand(m, 16, seed=3) @ rand(16, n, seed=4) + 0.05 * rand(m, n, seed=5)
    got = sg.orthogonalize(g.cuda())
    check(got, plain(g), 5)
    # the part of the result outside the strong directions
    u = torch.linalg.qr(g.double() @ rand(n, 16, seed=6).double()).Q
    w, x = plain(g), got.cpu().double()
    rest = lambda t: t - u @ (u.T @ t)  # noqa: E731
    assert (rest(x) - rest(w)).norm() <= 10 * tolerance(5, torch.float32) * rest(w).norm()


@pytest.mark.parametrize("magnitude", [1e-42, 1e-30, 1e-4, 1e30, 1e37])
@pytest.mark.parametrize("shape", [(50, 70), (200, 150)], ids=lambda s: "x".join(map(str, s)))
def test_magnitudes(shape, magnitude):
    g = rand(*shape, seed=7) * magnitude
    check(sg.orthogonalize(g.cuda(), eps=0.0), plain(g, eps=0.0), 5)


def test_eps_is_added_to_the_norm():
    g = rand(40, 60, seed=8) * 1e-8
    check(sg.orthogonalize(g.cuda(), eps=1e-6), plain(g, eps=1e-6), 5)


def test_zero_matrices():
    for eps in (0.0, 1e-7):
        assert (sg.orthogonalize(torch.zeros(70, 30, device="cuda"), eps=eps) == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_stays_in_its_matrix(bad):
    g = rand(3, 140, 200, seed=9)
    want = sg.orthogonalize(g.cuda())
    g[1, 77, 3] = bad
    got = sg.orthogonalize(g.cuda())
    assert torch.isnan(got[1]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("gtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("otype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(100, 140), (140, 100)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("steps", [0, 5])
def test_alpha_beta_is_the_whole_update(shape, gtype, otype, steps):
    g = rand(*shape, seed=10).to(gtype)
    w = rand(*shape, seed=11).to(otype)
    wide = torch.full((shape[0] + 2, shape[1] + 9), 5.0, dtype=otype, device="cuda")
    view = wide[1:-1, 4:-5]
    view.copy_(w)
    got = sg.orthogonalize(g.cuda(), steps=steps, alpha=-0.25, beta=0.5, out=view)
    assert got is view
    x = plain(g, steps)
    want = 0.5 * w.double() - 0.25 * x
    tol = 0.25 * tolerance(steps, torch.float32) * x.norm() + ROUND[otype] * want.norm()
    assert (view.cpu().double() - want).norm() <= tol
    wide[1:-1, 4:-5] = 5.0
    assert (wide == 5.0).all()


def test_strides_and_in_place():
    buf = torch.full((4, 90, 300), float("nan")).cuda()
    view = buf[1:3, 5:85, 3:253]
    g = rand(2, 80, 250, seed=12)
    view.copy_(g)
    check(sg.orthogonalize(view), plain(g), 5)
    assert sg.orthogonalize(view, out=view) is view
    check(view, plain(g), 5)
    assert torch.isnan(buf[0]).all() and torch.isnan(buf[1:3, :5]).all()
    assert torch.isnan(buf[1:3, 5:85, 253:]).all()


def test_other_coefficients_reach_the_orthogonal_factor():
    """x (3 - x^2) / 2 converges to 1 from any x in (0, sqrt 3): the rows become orthonormal."""
    g = torch.eye(90, 150) + 0.02 * rand(90, 150, seed=13)
    x = sg.orthogonalize(g.cuda(), steps=20, coefficients=(1.5, -0.5, 0.0)).cpu().double()
    u, _, v = torch.linalg.svd(g.double(), full_matrices=False)
    # at the fixed point the map no longer stretches errors along the singular directions
    assert (x - u @ v).abs().max() <= 64 * EPS
    assert (x @ x.T - torch.eye(90)).abs().max() <= 64 * EPS


@pytest.mark.parametrize("coefficients", [(50.0, 0.0, 0.0), (1e-3, 0.0, 0.0), (0.0, 3.0, 0.0),
                                          (2.0, 0.0, -40.0), (0.0, 0.0, 0.0)])
def test_results_far_from_one(coefficients):
    g = torch.diag(torch.linspace(0.2, 1.0, 40)) + 0.01 * rand(40, 40, seed=14)
    a, b, c = coefficients
    x = plain(g, 1, coefficients)
    got = sg.orthogonalize(g.cuda(), steps=1, coefficients=coefficients).cpu().double()
    size = (abs(a) + abs(b) + abs(c)) * (g.double() / g.double().norm()).norm()
    assert (got - x).norm() <= EPS * size
    if coefficients == (2.0, 0.0, -40.0):  # 38, 3e9, 1e49: norms up to that are possible
        with pytest.raises(sg.SgemmError) as e:
            sg.orthogonalize(g.cuda(), steps=3, coefficients=coefficients)
        assert e.value.status == -9
    else:
        assert torch.isfinite(sg.orthogonalize(g.cuda(), steps=3, coefficients=coefficients)).all()


def test_same_bits_every_time():
    g = rand(2, 300, 900, seed=15).cuda()
    first = sg.orthogonalize(g)
    for _ in range(5):
        assert torch.equal(first, sg.orthogonalize(g))


def test_another_stream_and_a_graph():
    g = rand(200, 333, seed=16).cuda()
    want = sg.orthogonalize(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = sg.orthogonalize(g)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sg.orthogonalize(g)
    g.copy_(rand(200, 333, seed=17))
    graph.replay()
    torch.cuda.synchronize()
    check(got, plain(g.cpu()), 5)


def test_large_against_the_iteration_on_the_gpu():
    g = rand(1500, 2200, seed=18).cuda()
    check(sg.orthogonalize(g), plain(g).cpu(), 5)


def test_empty():
    for shape in ((0, 5), (5, 0), (0, 4, 4), (2, 0, 4)):
        assert sg.orthogonalize(torch.empty(shape, device="cuda")).shape == shape


def test_refusals_on_the_gpu():
    g = torch.zeros(4, 6, device="cuda")
    with pytest.raises(TypeError):
        sg.orthogonalize(g.double())
    with pytest.raises(ValueError):
        sg.orthogonalize(g[0])
    with pytest.raises(ValueError):
        sg.orthogonalize(g.t())
    with pytest.raises(ValueError):
        sg.orthogonalize(g, out=torch.zeros(4, 5, device="cuda"))
    with pytest.raises(ValueError):
        sg.orthogonalize(g, beta=1.0)
    with pytest.raises(TypeError):
        sg.orthogonalize(g, out=g, out_dtype=torch.bfloat16)
    for kw, code in ((dict(steps=65), -8), (dict(coefficients=(1e9, 0.0, 0.0)), -9),
                     (dict(coefficients=(float("nan"), 0.0, 0.0)), -9), (dict(eps=-1.0), -10)):
        with pytest.raises(sg.SgemmError) as e:
            sg.orthogonalize(g, **kw)
        assert e.value.status == code


@pytest.mark.parametrize("otype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(20, 300), (256, 256), (300, 1100), (700, 520), (4, 300, 300)],
                         ids=lambda s: "x".join(map(str, s)))
def test_16_bit_results_are_the_fp32_ones_rounded_once(shape, otype):
    """The type of the result changes its last rounding, and nothing that comes before it."""
    g = rand(*shape, seed=19).to(otype).cuda()
    wide = sg.orthogonalize(g, out_dtype=torch.float32)
    assert torch.equal(sg.orthogonalize(g), wide.to(otype))
    out = rand(*shape, seed=20).to(otype).cuda()
    want = torch.addcmul(0.5 * wide, out.float(), torch.tensor(-2.0, device="cuda")).to(otype)
    assert torch.equal(sg.orthogonalize(g, alpha=0.5, beta=-2.0, out=out), want)


def test_overlapping_rows_are_refused():
    g = torch.zeros(8, 60, device="cuda")
    for bad in (g[:1].expand(8, 60), torch.zeros(67, device="cuda").unfold(0, 60, 1)):
        with pytest.raises(ValueError, match="overlap"):
            sg.orthogonalize(bad)
        with pytest.raises(ValueError, match="overlap"):
            sg.orthogonalize(g, out=bad)


@pytest.mark.parametrize("shape", [(1, 20, 3000), (1, 32, 16), (1, 16, 16), (1, 2048, 16), (1, 128, 1000),
                                   (60, 32, 16), (40, 20, 3000)], ids=lambda s: "x".join(map(str, s)))
def test_narrow_matrices_are_as_exact_as_plain_32_bit_products(shape):
    """Mean error over matrices with a few strong directions and without. A short side has few sums to
    average the rounding of 22-bit factors out; a twentieth more is left for the mean of so few."""
    def steps_in(x, eps=1e-7):
        tall = x.shape[-2] > x.shape[-1]
        x = x.mT if tall else x
        x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + eps)
        for _ in range(5):
            s = x @ x.mT
            x = USUAL[0] * x + (USUAL[1] * s + USUAL[2] * (s @ s)) @ x
        return x.mT if tall else x

    ours, products = [], []
    for seed in range(8):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        g = torch.randn(*shape, generator=gen, device="cuda")
        b, m, n = shape
        r = max(1, min(m, n) // 16)
        u, v = (torch.randn(b, *s, generator=gen, device="cuda") for s in ((m, r), (r, n)))
        for x in (g, 1e-3 * (g + u @ v)):
            w = steps_in(x.double())
            norm = w.square().sum(dim=(1, 2)).sqrt()
            for got, errors in ((sg.orthogonalize(x), ours), (steps_in(x), products)):
                errors += ((got.double() - w).square().sum(dim=(1, 2)).sqrt() / norm).tolist()
    assert sum(ours) <= 1.05 * sum(products), (sum(ours) / len(ours), sum(products) / len(products))


@pytest.mark.parametrize("steps", [0, 1])
def test_more_matrices_than_a_grid_has_rows(steps):
    """65537 and more matrices; 6 x 2 and 2 x 6 padded to 128 x 128."""
    for shape in ((65538, 2, 6), (65538, 6, 2)):
        g = torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
        got = sg.orthogonalize(g, steps=steps).double()
        want = plain(g, steps)
        err = (got - want).square().sum(dim=(1, 2)).sqrt()
        assert (err <= tolerance(steps, torch.float32) * want.square().sum(dim=(1, 2)).sqrt()).all()
