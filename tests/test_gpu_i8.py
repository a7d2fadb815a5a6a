"""GPU tests of the linear layer on 8-bit integers and its quantiser against 64-bit forms.

Quantiser: equality, bit for bit: both divisions are rounded once and the product with 127 / a is exact
until it is rounded to a whole number.

Product: the sum over k is a whole number that no kernel may miss, so with scales that are powers of two
results are equal to it, rounded once to the type (in FP32, then in it: a sum past 2^24 is rounded twice
on its way to 16 bits). With other scales, u = 2^-24: the sum's rounding, the two scales' product and the
multiply-add are within u each, so that D is within 3 u |sums| + u |D| + 2 u |beta D0|, and half a step
of its type.
"""
import pytest
import torch

from i8_plans import SHAPES as PLANS

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

U = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


@pytest.fixture(autouse=True)
def status_clear():
    yield
    assert sg.i8_linear_status() == (0, 0)


# ------------------------------------------------------------------------------ quantiser

def plain_quantize(x):
    x = x.double().cpu()
    a = x.abs().amax(1, keepdim=True).clamp_min(2.0 ** -119)

    def f32(t):  # a quotient rounded to 53 bits first rounds to the same FP32 number
        return t.float().double()

    return torch.round(x * f32(127.0 / a)).to(torch.int8), f32(a / 127.0)[:, 0].float()


def check_quantized(x, q, s):
    eq, es = plain_quantize(x)
    assert q.dtype == torch.int8 and s.dtype == torch.float32 and q.shape == x.shape and s.shape == x.shape[:1]
    assert torch.equal(s.cpu(), es)
    assert torch.equal(q.cpu(), eq)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1), (1, 16), (3, 64), (70, 65), (5, 256), (300, 257), (7, 512), (33, 777),
                                   (9, 1024), (4, 1025), (5, 2048), (3, 2056), (1, 4096), (3, 4100), (2, 8192),
                                   (3, 8200), (2, 16384), (2, 16392), (1, 40001)],
                         ids=lambda s: "x".join(map(str, s)))
def test_quantize(shape, dtype):
    x = (rand(*shape, seed=shape[1]) * torch.exp(2 * rand(shape[0], 1, seed=1))).to(dtype).cuda()
    check_quantized(x, *sg.i8_quantize(x))


@pytest.mark.parametrize("shape", [(20000, 40), (9000, 200), (3000, 1500), (2500, 4096), (700, 16000), (400, 20000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_quantize_many_rows(shape):
    x = rand(*shape, seed=4).to(torch.bfloat16).cuda()
    check_quantized(x, *sg.i8_quantize(x))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(2500, 1000), (620, 4608), (620, 6144), (620, 6145), (310, 8193), (310, 12288),
                                   (310, 12289), (160, 16384)], ids=lambda s: "x".join(map(str, s)))
def test_quantize_layouts_of_long_rows(shape, dtype):
    x = (rand(*shape, seed=9) * torch.exp(2 * rand(shape[0], 1, seed=1))).to(dtype).cuda()
    check_quantized(x, *sg.i8_quantize(x))


@pytest.mark.parametrize("cols", [33, 390, 4000, 17000])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_strided_and_unaligned(cols, offset, dtype):
    buf = torch.full((9, cols + 11), float("nan"), dtype=dtype, device="cuda")
    view = buf[2:7, offset:offset + cols]
    view.copy_(rand(5, cols, seed=5))
    check_quantized(view, *sg.i8_quantize(view))


@pytest.mark.parametrize("cols", [256, 3000, 20000])
def test_quantize_extremes(cols):
    """Zero rows, the smallest and the largest numbers, ties of the rounding."""
    x = torch.zeros(8, cols)
    x[1, 3] = 1e-45
    x[2, 5], x[2, 6] = 3.4e38, -3.4e38
    x[3, :10] = 2.0 ** -119 * torch.arange(10)
    x[4, :255] = torch.arange(-127, 128) * 0.5 + 0.5  # every tie, with 127 / a = 1 below
    x[4, 200] = 127.0
    x[5, :255] = torch.arange(-127, 128).float()
    x[6] = rand(cols, seed=6) * 1e-38
    x[7] = -5.0
    check_quantized(x.cuda(), *sg.i8_quantize(x.cuda()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [64, 3000, 20000])
def test_quantize_not_finite(cols, dtype):
    x = rand(6, cols, seed=6).to(dtype)
    x[1, 7], x[4, cols - 1], x[5, 0] = float("nan"), float("-inf"), float("inf")
    q, s = sg.i8_quantize(x.cuda())
    for r in range(6):
        if r in (1, 4, 5):
            assert torch.isnan(s[r]) and (q[r] == 0).all()
        else:
            check_quantized(x[r:r + 1], q[r:r + 1], s[r:r + 1])


@pytest.mark.parametrize("shape", [(0, 5), (5, 0), (0, 0)])
def test_quantize_empty(shape):
    q, s = sg.i8_quantize(torch.empty(shape, device="cuda"))
    assert q.shape == shape and s.shape == shape[:1]
    assert torch.equal(s.cpu(), plain_quantize(torch.zeros(shape[0], 1))[1])


def test_quantize_leaves_the_padding():
    x = rand(5, 100, seed=7).cuda()
    q = torch.full((5, 112), 0x5a, dtype=torch.int8, device="cuda")
    s = torch.empty(5, device="cuda")
    assert sg.lib.i8_quantize(5, 100, x.data_ptr(), 0, 100, q.data_ptr(), 112, s.data_ptr(),
                              torch.cuda.current_stream().cuda_stream or None) == 0
    assert (q[:, 100:] == 0x5a).all()
    check_quantized(x, q[:, :100], s)


def test_quantize_offsets_past_32_bits():
    rows, cols = 66048, 65664
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(cols, device="cuda").to(torch.bfloat16)
    q, s = sg.i8_quantize(x)
    check_quantized(x[-1:], q[-1:], s[-1:])
    x = x.view(-1)[:1 << 32].view(1 << 20, 4096)
    x[-1] = torch.arange(4096, device="cuda").to(torch.bfloat16)
    q, s = sg.i8_quantize(x)
    check_quantized(x[-1:], q[-1:], s[-1:])


# ------------------------------------------------------------------------------ product

def stored(q, extra=0):
    """On the GPU in rows of a multiple of 16 bytes, with other bytes between them."""
    rows, cols = q.shape
    held = torch.full((rows, (cols + 15) // 16 * 16 + extra), 0x55, dtype=torch.int8, device="cuda")
    held[:, :cols] = q.cuda()
    return held[:, :cols]


def whole(rows, cols, seed, low=-128, high=127):
    return torch.randint(low, high + 1, (rows, cols), dtype=torch.int8, generator=torch.Generator().manual_seed(seed))


def sums(x, w):
    return x.cuda().double() @ w.cuda().double().t()  # (exact: far below 2^53)


def check(M, N, K, dtype=torch.float32, bias=False, beta=0.0, seed=0, extra=0):
    x, w = stored(whole(M, K, seed), extra), stored(whole(N, K, seed + 1), extra)
    want = sums(x, w)
    one, quarter = torch.ones(M, device="cuda"), torch.full((N,), 0.25, device="cuda")
    exact = sg.i8_linear(x, one, w, quarter, out_dtype=dtype)
    assert exact.dtype == dtype and exact.shape == (M, N)
    assert torch.equal(exact, (want.float() * 0.25).to(dtype))
    sx, sw = torch.exp(rand(M, seed=seed + 2)).cuda() / 200, torch.exp(rand(N, seed=seed + 3)).cuda() / 200
    b = rand(N, seed=seed + 4).cuda() if bias else None
    old = rand(M, N, seed=seed + 5).to(dtype).cuda() if beta else None
    got = sg.i8_linear(x, sx, w, sw, b, beta=beta, out=None if old is None else old.clone(), out_dtype=dtype)
    product = want * sx.double()[:, None] * sw.double()
    D = product + (b.double() if bias else 0) + (beta * old.double() if beta else 0)
    tol = 3 * U * product.abs() + U * D.abs() + (2 * U * (beta * old.double()).abs() if beta else 0)
    tol = tol + torch.finfo(dtype).eps / 2 * (D.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0)
    if bias or beta:
        tol = tol + 2 * U * (D - product).abs()
    assert ((got.double() - D).abs() <= tol).all()


SHAPES = ([(m, 260, 333) for m in (1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 129, 200)]
          + [(m, n, 272) for m in (1, 6, 12, 40, 150) for n in (1, 2, 31, 127, 128, 129, 383)]
          + [(m, 130, k) for m in (1, 5, 20, 140) for k in (1, 2, 15, 16, 17, 127, 128, 129, 1024, 1025, 2047, 2049)]
          + [(300, 700, 1000), (517, 301, 777), (1000, 130, 1200), (9, 3001, 2000), (64, 2000, 5000)])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product_shapes(shape):
    check(*shape, bias=shape[0] % 2 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("plan", PLANS, ids=lambda p: "-".join(map(str, p)))
def test_product_every_plan(plan, dtype):
    """Each tile and split, with a result at any alignment, one that is added to, and a bias."""
    M, N, K = PLANS[plan]
    check(M, N, K, dtype=dtype, bias=True)
    check(M, N + 7, K, dtype=dtype, beta=0.5, extra=48)


@pytest.mark.parametrize("shape", [(2600, 2700, 300), (2305, 4400, 1100), (2433, 4353, 129), (3000, 130, 3000),
                                   (200, 5000, 2000)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product_large(shape, dtype):
    """Several tiles for each block, pairs of blocks."""
    check(*shape, dtype=dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bias,beta", [(False, 0.0), (True, 0.0), (False, 1.0), (True, -0.5)])
@pytest.mark.parametrize("shape", [(1, 300, 100), (7, 301, 700), (20, 300, 2000), (60, 257, 200), (150, 301, 270),
                                   (2050, 2100, 140)], ids=lambda s: "x".join(map(str, s)))
def test_product_types_bias_beta(shape, dtype, bias, beta):
    check(*shape, dtype=dtype, bias=bias, beta=beta, extra=16)


@pytest.mark.parametrize("value", [(127, 127), (-128, -128), (-128, 127)])
@pytest.mark.parametrize("shape", [(1, 130, 5000), (8, 130, 131071), (9, 130, 131071), (30, 260, 4096), (64, 128, 3000),
                                   (130, 130, 131071), (2304, 2560, 3000)], ids=lambda s: "x".join(map(str, s)))
def test_product_largest_sums(shape, value):
    """Sums of equal products: no accumulator may round, and 32 bits hold them all."""
    M, N, K = shape
    x, w = stored(torch.full((M, K), value[0], dtype=torch.int8)), stored(torch.full((N, K), value[1], dtype=torch.int8))
    y = sg.i8_linear(x, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), out_dtype=torch.float32)
    assert (y == float(torch.tensor(float(K * value[0] * value[1])))).all()


@pytest.mark.parametrize("M", [3, 12, 30, 60, 140, 2304])
def test_product_sums_near_the_accumulators_limit(M):
    """Large products of one sign and small ones of the other, in every order."""
    N, K = (2560 if M > 2000 else 256), 2048
    x, w = whole(M, K, 1, 100, 127), whole(N, K, 2, 100, 127)
    for k in range(0, K, 7):
        w[:, k] = whole(N, 1, k, -3, 3)[:, 0]
    x, w = stored(x), stored(w)
    one = torch.ones(max(M, N), device="cuda")
    want = sums(x, w)
    assert want.abs().max() > 1 << 24
    got = sg.i8_linear(x, one[:M], w, one[:N], out_dtype=torch.float32)
    assert torch.equal(got, want.float())
    # the last bits too: the largest part of each sum taken out by the result that is there
    base = (want / 4096).floor() * 4096
    got = sg.i8_linear(x, one[:M], w, one[:N], beta=-1.0, out=base.float())
    assert ((got.double() - (want - base)).abs() <= 4).all()


def test_product_views():
    """D as a view into a larger matrix, whose other elements are left alone, at any alignment."""
    for M, N, K in ((3, 100, 200), (40, 131, 300), (200, 301, 150)):
        x, w = stored(whole(M, K, 1), 32), stored(whole(N, K, 2), 16)
        sx, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        for dtype in TYPES:
            want = sg.i8_linear(x, sx, w, sw, out_dtype=dtype)
            for offset in (0, 1, 2, 8):
                buf = torch.full((M + 2, N + 13), float("nan"), dtype=dtype, device="cuda")
                out = buf[1:-1, offset:offset + N]
                assert sg.i8_linear(x, sx, w, sw, out=out) is out
                assert torch.equal(out, want)
                out.fill_(float("nan"))
                assert torch.isnan(buf).all()


@pytest.mark.parametrize("M", [2, 20, 140])
def test_product_not_finite_scales_stay_where_they_belong(M):
    x, w = stored(whole(M, 200, 1)), stored(whole(150, 200, 2))
    sx, sw = torch.rand(M, device="cuda"), torch.rand(150, device="cuda")
    want = sg.i8_linear(x, sx, w, sw)
    sx[1], sw[140] = float("nan"), float("nan")
    got = sg.i8_linear(x, sx, w, sw)
    bad = torch.isnan(got)
    assert bad[1].all() and bad[:, 140].all() and bad.sum() == 150 + M - 1
    assert torch.equal(got[~bad], want[~bad])


def test_product_empty():
    for M, N in ((0, 5), (5, 0), (0, 0)):
        y = sg.i8_linear(stored(whole(M, 20, 1)), torch.ones(M, device="cuda"), stored(whole(N, 20, 2)),
                         torch.ones(N, device="cuda"))
        assert y.shape == (M, N)
    x, w = torch.empty(30, 0, dtype=torch.int8, device="cuda"), torch.empty(40, 0, dtype=torch.int8, device="cuda")
    sx, sw, b = torch.ones(30, device="cuda"), torch.ones(40, device="cuda"), rand(40, seed=1).cuda()
    assert (sg.i8_linear(x, sx, w, sw) == 0).all()
    y = torch.ones(30, 40, device="cuda")
    sg.i8_linear(x, sx, w, sw, b, beta=2.0, out=y)
    assert torch.equal(y, (b + 2).expand(30, 40))


@pytest.mark.parametrize("shape", [(1, 14336, 4096), (16, 4096, 8192), (100, 4096, 4096), (700, 3000, 2000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_cold_weights_back_to_back(shape):
    """Weights from memory, not from the cache: copies of neighbouring k blocks land in any order."""
    M, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    ws = [torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8) for _ in range(6)]
    one = torch.ones(max(M, N), device="cuda")
    want = [sums(x, w).float() for w in ws]
    for _ in range(10):
        got = [sg.i8_linear(x, one[:M], w, one[:N], out_dtype=torch.float32) for w in ws]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_chain_on_another_stream_and_in_a_graph():
    w, b = sg.i8_quantize(rand(500, 700, seed=2).cuda()), rand(500, seed=3).cuda()
    for M in (1, 24, 300):
        x = rand(M, 700, seed=M).to(torch.bfloat16).cuda()

        def chain():
            return sg.i8_linear(*sg.i8_quantize(x), *w, b)

        want = chain()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = chain()
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain()
        x.mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, sg.i8_linear(*sg.i8_quantize(x), *w, b))
        assert not torch.equal(got, want)


def test_product_offsets_past_32_bits():
    """D and the operands past 2^31 and 2^32 elements: sampled rows and columns."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def some(rows, cols):
        return torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)

    for M, N, K in ((66048, 65664, 128), (5, 1100000, 4096), (40, 1100000, 4096), (1100000, 300, 4096)):
        x, w = some(M, K), some(N, K)
        one = torch.ones(max(M, N), device="cuda")
        d = sg.i8_linear(x, one[:M], w, one[:N], out_dtype=torch.float32)
        for r in {0, M // 2, M - 1}:
            for c in (0, max(0, N // 2 - 50), max(0, N - 100)):
                assert torch.equal(d[r, c:c + 100], sums(x[r:r + 1], w[c:c + 100])[0].float())
        del x, w, d


def test_refusals_on_the_gpu():
    q = torch.zeros(64, 160, dtype=torch.int8, device="cuda")
    s = torch.ones(64, device="cuda")
    assert sg.i8_linear(q, s, q, s).dtype == torch.bfloat16
    with pytest.raises(ValueError):  # one scale for each row
        sg.i8_linear(q, s[:63], q, s)
    with pytest.raises(ValueError):
        sg.i8_linear(q, s, q, s[:, None])
    with pytest.raises(ValueError):
        sg.i8_linear(q, torch.ones(128, device="cuda")[::2], q, s)
    with pytest.raises(TypeError):
        sg.i8_linear(q, s.half(), q, s)
    with pytest.raises(TypeError):
        sg.i8_linear(q, s, q.view(torch.uint8), s)
    with pytest.raises(ValueError):  # inner sizes
        sg.i8_linear(q, s, q[:, :128], s)
    with pytest.raises(ValueError):  # k is not contiguous
        sg.i8_linear(q, s, torch.zeros(160, 64, dtype=torch.int8, device="cuda").t(), s)
    with pytest.raises(ValueError, match="overlap"):
        sg.i8_linear(q[:1].expand(64, 160), s, q, s)
    with pytest.raises(ValueError):  # beta without out
        sg.i8_linear(q, s, q, s, beta=1.0)
    with pytest.raises(ValueError):
        sg.i8_linear(q, s, q, s, s[:5])
    with pytest.raises(TypeError):
        sg.i8_linear(q, s, q, s, s.half())
    with pytest.raises(TypeError):
        sg.i8_linear(q, s, q, s, out=torch.zeros(64, 64, device="cuda").double())
    with pytest.raises(ValueError):
        sg.i8_linear(q, s, q, s, out=torch.zeros(64, 65, device="cuda"))
    for bad, code in ((q[:, 1:], -4), (torch.zeros(64, 24, dtype=torch.int8, device="cuda"), -5)):
        with pytest.raises(sg.SgemmError) as e:
            sg.i8_linear(bad, s, bad, s)
        assert e.value.status == code
    with pytest.raises(sg.SgemmError) as e:
        t = torch.zeros(1, 1 << 17, dtype=torch.int8, device="cuda")
        sg.i8_linear(t, s[:1], t, s[:1])
    assert e.value.status == -3
