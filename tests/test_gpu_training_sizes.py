"""GPU tests of the 8-bit product and the orthogonalisation at the sizes of an MLP's weight, and of
orthogonalisations beside other work on the GPU. Bounds as in test_gpu_f8.py and
test_gpu_orthogonalize.py; 64-bit forms on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

U32, U16 = 2.0 ** -23, 2.0 ** -8


@pytest.fixture(autouse=True)
def status_clear():
    yield
    assert sg.f8_gemm_status() == (0, 0) and sg.ns_orthogonalize_status() == (0, 0)


def rand(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return scale * torch.randn(*shape, generator=g, device="cuda")


def values(q, s, block):
    br, bc = block
    rows, cols = q.shape
    return q.double() * s.double().repeat_interleave(br, 0)[:rows].repeat_interleave(bc, 1)[:, :cols]


# (tokens, outputs, inputs): contractions over 14336 and more in each of the three products
@pytest.mark.parametrize("tokens,outputs,inputs", [(1, 4096, 14336), (16, 4096, 14336), (33, 520, 28671),
                                                   (1024, 4096, 14336)])
def test_long_contractions_forward(tokens, outputs, inputs):
    x, w = rand(tokens, inputs, seed=1).bfloat16(), rand(outputs, inputs, seed=2)
    q, s = sg.f8_quantize(x)
    wq, ws = sg.f8_quantize(w, (128, 128))
    a, b = values(q, s, (1, 128)), values(wq, ws, (128, 128))
    R, S = a @ b.t(), a.abs() @ b.abs().t()
    for dtype, u in ((torch.float32, U32), (torch.bfloat16, U16)):
        y = sg.f8_matmul(q, s, wq, ws, transb=True, out_dtype=dtype)
        assert ((y.double() - R).abs() <= (inputs + 8) * U32 * S + u * R.abs()).all()


def test_long_contractions_backward():
    tokens, outputs, inputs = 14337, 1100, 700
    dy, x = rand(tokens, outputs, seed=3, scale=1e-5).bfloat16(), rand(tokens, inputs, seed=4).bfloat16()
    dyc, xc = sg.f8_quantize(dy, (128, 1), dtype=torch.float8_e5m2), sg.f8_quantize(x, (128, 1))
    a, b = values(*dyc, (128, 1)), values(*xc, (128, 1))
    grad = rand(outputs, inputs, seed=5, scale=1e-4)
    R = grad.double() + a.t() @ b
    S = a.abs().t() @ b.abs() + grad.double().abs()
    sg.f8_matmul(*dyc, *xc, transa=True, beta=1.0, out=grad)
    assert ((grad.double() - R).abs() <= (tokens + 9) * U32 * S).all()
    # the input gradient over 14336 outputs
    dy, w = rand(300, 14336, seed=6, scale=1e-5).bfloat16(), rand(14336, 700, seed=7)
    q, wq = sg.f8_quantize(dy), sg.f8_quantize(w, (128, 128))
    a, b = values(*q, (1, 128)), values(*wq, (128, 128))
    R = a @ b
    dx = sg.f8_matmul(*q, *wq)
    assert ((dx.double() - R).abs() <= 14344 * U32 * (a.abs() @ b.abs()) + U16 * R.abs()).all()


def iterate(g, steps):
    a, b, c = 3.4445, -4.7750, 2.0315
    tall = g.shape[-2] > g.shape[-1]
    x = g.double().mT if tall else g.double()
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + 1e-7)
    for _ in range(steps):
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.mT if tall else x


@pytest.mark.parametrize("shape,dtype,steps", [
    ((4096, 14336), torch.float32, 2), ((14336, 4096), torch.bfloat16, 2),
    ((1024, 16384), torch.float32, 5), ((4096, 4096), torch.float32, 2),
    ((8, 1024, 1024), torch.bfloat16, 5), ((8, 1024, 1024), torch.float32, 5),
    ((4097, 777), torch.float32, 5), ((4097, 777), torch.bfloat16, 5), ((2, 2200, 1500), torch.float16, 3),
], ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v).split(".")[-1])
def test_large_updates(shape, dtype, steps):
    g = rand(*shape, seed=8).to(dtype)
    x = iterate(g, steps)
    bound = 2.0 ** -20 * sum(4.0 ** k for k in range(steps))
    u = {torch.float32: U32, torch.bfloat16: U16, torch.float16: 2.0 ** -11}[dtype]
    got = sg.orthogonalize(g, steps=steps)
    assert (got.double() - x).norm() <= (bound + u) * x.norm()
    w = rand(*shape, seed=9)
    want = 0.75 * w.double() - 0.125 * x
    sg.orthogonalize(g, steps=steps, alpha=-0.125, beta=0.75, out=w)
    assert (w.double() - want).norm() <= 0.125 * (bound + U32) * x.norm() + U32 * want.norm()


@pytest.mark.parametrize("shapes", [
    [(256, 256), (300, 200)],                        # both fit on the GPU side by side
    [(4097, 777), (256, 256), (1024, 1024)],         # the larger ones take all of it
    [(1163, 1928), (8, 642, 772), (771, 1301)],      # pairs of blocks and single ones
], ids=["small", "mixed", "pairs"])
def test_updates_on_several_streams_beside_products(shapes):
    """Each update's blocks wait for one another: they have to be on the GPU together, whatever else
    the other streams put there."""
    gs = [rand(*shape, seed=20 + i) for i, shape in enumerate(shapes)]
    x, w = rand(4096, 2048, seed=30).bfloat16(), rand(4096, 2048, seed=31)
    q, wq = sg.f8_quantize(x), sg.f8_quantize(w, (128, 128))
    one = sg.f8_quantize(x[:1])
    want = [sg.orthogonalize(g) for g in gs]
    want_y, want_one = sg.f8_matmul(*q, *wq, transb=True), sg.f8_matmul(*one, *wq, transb=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(len(gs) + 2)]
    got, ys, ones = [[] for _ in gs], [], []
    for _ in range(10):
        for g, results, stream in zip(gs, got, streams):
            with torch.cuda.stream(stream):
                results.append(sg.orthogonalize(g))
        with torch.cuda.stream(streams[-2]):
            ys.append(sg.f8_matmul(*q, *wq, transb=True))
        with torch.cuda.stream(streams[-1]):
            ones += [sg.f8_matmul(*one, *wq, transb=True) for _ in range(5)]
    torch.cuda.synchronize()
    for results, w in zip(got, want):
        assert all(torch.equal(r, w) for r in results)
    assert all(torch.equal(y, want_y) for y in ys) and all(torch.equal(y, want_one) for y in ones)
