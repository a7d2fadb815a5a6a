"""GPU tests of the norm of all gradients and of clipping by it, against 64-bit forms.

Bounds, with u = 2^-24: a square and the 64 additions of a thread's sum are within 66 u of the exact
sum relative to it, the rest is 64-bit, the root halves that and the norm is rounded once: 35 u. A
clipped element is off by the factor's 35 u and its rounding u, the product's u, and the rounding to its
type (half a step; 2^-25 more in FP16).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

U = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]
EPS = 1e-6


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def exact(grads, max_norm, eps=EPS):
    norm = math.sqrt(sum(g.double().square().sum().item() for g in grads))
    return norm, min(1.0, max_norm / (norm + eps)) if norm else 1.0


def check(grads, max_norm, norm, out, eps=EPS):
    want, factor = exact(grads, max_norm, eps)
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(norm.item() - want) <= 35 * U * want
    for g, o in zip(grads, out):
        w = g.double() * factor
        tol = (38 * U + torch.finfo(o.dtype).eps / 2) * w.abs() + (2.0 ** -25 if o.dtype == torch.float16 else 0)
        assert o.shape == g.shape and ((o.double() - w).abs() <= tol).all()


def problem(sizes, types, seed=0):
    return [(rand(n, seed=seed + i) * math.exp(0.3 * (i % 5))).to(types[i % len(types)]).cuda()
            for i, n in enumerate(sizes)]


SIZES = [[1], [7], [16384], [16385, 3], [100000], [5, 0, 64, 1, 0, 17, 33000, 2], [0, 0, 9], [1 << 20, 12345]]


@pytest.mark.parametrize("max_norm", [0.5, 1e9])
@pytest.mark.parametrize("types", [[t] for t in TYPES] + [TYPES], ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_sizes(sizes, types, max_norm):
    grads = problem(sizes, types)
    before = [g.clone() for g in grads]
    for kinds in (types, TYPES[::-1]):  # results of the same and of other types
        out = [torch.full_like(g, float("nan"), dtype=kinds[i % len(kinds)]) for i, g in enumerate(grads)]
        check(grads, max_norm, sg.clip_grad_norm(grads, max_norm, out=out), out)
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    norm = sg.clip_grad_norm(grads, max_norm)
    check(before, max_norm, norm, grads)
    if max_norm == 1e9:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))


@pytest.mark.parametrize("count", [95, 96, 97, 961, 2000])
def test_many_arrays(count):
    """One table of arrays, the largest ones, and several."""
    sizes = [(i * 37) % 300 + (20000 if i % 100 == 3 else 0) for i in range(count)]
    grads = problem(sizes, TYPES)
    before = [g.clone() for g in grads]
    check(before, 3.0, sg.clip_grad_norm(grads, 3.0), grads)


def test_shapes_and_views():
    """Matrices and scalars, and neighbouring pieces of one buffer that begin anywhere."""
    buf = rand(100001, seed=3).cuda()
    before = buf.clone()
    cuts = [1, 2, 5, 1000, 1003, 40000, 100000]
    grads = [buf[a:b] for a, b in zip(cuts, cuts[1:])]
    grads[4:5] = [grads[4][:38990].view(10, 3899)]
    want, factor = exact(grads, 2.0)
    norm = sg.clip_grad_norm(grads, 2.0)
    assert abs(norm.item() - want) <= 35 * U * want
    touched = torch.zeros_like(buf, dtype=torch.bool)
    touched[1:1003] = touched[1003:1003 + 38990] = touched[40000:100000] = True
    assert torch.equal(buf[~touched], before[~touched])
    assert ((buf - before * factor).abs()[touched] <= 40 * U * before.abs()[touched]).all()
    one = torch.tensor(3.0, device="cuda")
    assert sg.clip_grad_norm([one], 1.0, eps=0.0).item() == 3.0 and one.item() == 1.0


def test_only_the_norm():
    grads = problem([1000, 50], TYPES)
    before = [g.clone() for g in grads]
    norm = sg.clip_grad_norm(grads, float("inf"))
    check(before, 1e30, norm, grads)
    assert all(torch.equal(g, b) for g, b in zip(grads, before))
    out = [torch.empty_like(g, dtype=torch.float32) for g in grads]  # a conversion
    assert torch.equal(sg.clip_grad_norm(grads, float("inf"), out=out), norm)
    assert all(torch.equal(o, g.float()) for o, g in zip(out, grads))


@pytest.mark.parametrize("power", [-149, -130, -100, -75, -50, -40, 40, 55, 63, 100, 126])
def test_magnitudes(power):
    """Squares beyond FP32, in single pieces and next to others."""
    g = (1 + rand(40000, seed=1).abs()).cuda()
    a = g * 2.0 ** power if power > -140 else torch.full_like(g, 2.0 ** power)
    a = a.clamp(max=3e38)
    for grads in ([a], [a, g], [a[:5], g[:7]]):
        want, _ = exact(grads, 1.0)
        got = sg.clip_grad_norm(grads, float("inf")).item()
        if want > 3.4028235e38:
            assert got == math.inf
        else:  # (a denormal norm is good to its smallest step)
            assert abs(got - want) <= 35 * U * want + 2.0 ** -149
        out = [torch.empty_like(t) for t in grads]
        sg.clip_grad_norm(grads, 2.0 ** -20, eps=0.0, out=out)
        _, factor = exact(grads, 2.0 ** -20, 0.0)
        for o, t in zip(out, grads):
            w = t.double() * factor
            assert ((o.double() - w).abs() <= 40 * U * w.abs() + 2.0 ** -149).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite(bad):
    grads = problem([1000, 20000], [torch.float32])
    grads[1][7] = bad
    norm = sg.clip_grad_norm(grads, 1.0)
    if math.isnan(bad):
        assert torch.isnan(norm) and all(torch.isnan(g).all() for g in grads)
    else:
        assert norm.item() == math.inf and torch.isnan(grads[1][7])
        grads[1][7] = 0
        assert all((g == 0).all() for g in grads)


def test_zeros_and_none():
    grads = [torch.zeros(100, device="cuda"), torch.zeros(20000, device="cuda", dtype=torch.bfloat16)]
    for limit in (0.0, 1.0):
        assert sg.clip_grad_norm(grads, limit, eps=0.0).item() == 0.0
        assert all((g == 0).all() for g in grads)
    assert sg.clip_grad_norm([], 1.0).item() == 0.0
    assert sg.clip_grad_norm([torch.empty(0, device="cuda")], 1.0, out=[torch.empty(0, device="cuda")]).item() == 0.0
    g = problem([50], [torch.float32])
    assert sg.clip_grad_norm(g, 0.0).item() > 0 and (g[0] == 0).all()


def test_same_bits_every_time():
    grads = problem([3000000, 7, 555555, 20000], TYPES)
    out = [torch.empty_like(g) for g in grads]
    first = sg.clip_grad_norm(grads, 1.0, out=out)
    want = [o.clone() for o in out]
    for _ in range(3):
        assert torch.equal(sg.clip_grad_norm(grads, 1.0, out=out), first)
        assert all(torch.equal(o, w) for o, w in zip(out, want))


def test_past_32_bits():
    n = (1 << 32) + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-5:] = 4.0
    g[1 << 31] = 8.0
    want = math.sqrt(5 * 16 + 64)
    norm = sg.clip_grad_norm([g], 1.0, eps=0.0)
    assert abs(norm.item() - want) <= U * want * 2
    assert (g[-5:] == torch.tensor(4.0 / want).bfloat16().item()).all() and (g[-4000:-5] == 0).all()
    assert abs(g[1 << 31].item() - 8.0 / want) <= 2.0 ** -8


def test_another_stream_and_a_graph():
    grads = problem([5000, 300000, 3], TYPES)
    out = [torch.empty_like(g) for g in grads]
    want = sg.clip_grad_norm(grads, 1.0, out=out)
    clipped = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norm = sg.clip_grad_norm(grads, 1.0, out=out)
    side.synchronize()
    assert torch.equal(norm, want) and all(torch.equal(o, c) for o, c in zip(out, clipped))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = sg.clip_grad_norm(grads, 1.0, out=out)
    for g in grads:
        g.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, 2 * want)
    check(grads, 1.0, norm, out)


def test_refusals_on_the_gpu():
    g, h = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(TypeError):
        sg.clip_grad_norm([g, None], 1.0)
    with pytest.raises(TypeError):
        sg.clip_grad_norm([g.double()], 1.0)
    with pytest.raises(TypeError):
        sg.clip_grad_norm([g.cpu()], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        sg.clip_grad_norm([g[::2]], 1.0)
    with pytest.raises(ValueError):
        sg.clip_grad_norm([g], 1.0, out=[h[:5]])
    with pytest.raises(ValueError):
        sg.clip_grad_norm([g], 1.0, out=[h, h])
    for call, code in ((lambda: sg.clip_grad_norm([g, g], 1.0), -7),  # the same gradient twice
                       (lambda: sg.clip_grad_norm([g, g[60:]], 1.0), -7),
                       (lambda: sg.clip_grad_norm([g, h], 1.0, out=[h, g]), -7),
                       (lambda: sg.clip_grad_norm([g[:32], h[:32]], 1.0, out=[h[:32], h[32:]]), -7),
                       (lambda: sg.clip_grad_norm([g[:32]], 1.0, out=[g[8:40]]), -7),
                       (lambda: sg.clip_grad_norm([g], -1.0), -5),
                       (lambda: sg.clip_grad_norm([g], float("nan")), -5),
                       (lambda: sg.clip_grad_norm([g], 1.0, eps=-1.0), -6)):
        with pytest.raises(sg.SgemmError) as e:
            call()
        assert e.value.status == code
    assert (g == 1).all() and (h == 1).all()
    twice = sg.clip_grad_norm([g, g], float("inf"))  # read only: allowed
    assert twice.item() == pytest.approx(math.sqrt(128))
