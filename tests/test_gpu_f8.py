"""GPU tests of the 8-bit block-scaled product and its quantiser against plain 64-bit forms.

Quantiser: equality, bit for bit; scale and quotient are FP32 divisions, each correctly rounded,
and the last rounding goes to the nearest number of the format.

Product: with S = sum_k |a_k b_k| the error bound is
    |D - R| <= (K + 8) 2^-23 S            FP32 sums of K terms, each addition within 2^-23
                                          (the tensor core may truncate), scales and alpha
             + u |R| + 2^-23 |beta D0|    one rounding to D's type: u = 2^-23, 2^-8, 2^-11
and 2^-25 more for FP16, the spacing of its smallest numbers.
"""
import pytest
import torch

import f8_plain as plain

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
ROUND = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def rand(*shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * scale


@pytest.fixture(autouse=True)
def status_clear():
    yield
    assert sg.f8_gemm_status() == (0, 0)


# ------------------------------------------------------------------------------ quantiser

BLOCKS = [(1, 128), (128, 1), (128, 128)]


def check_quantized(x, block, dtype, pow2, q, s):
    eq, es = plain.quantize(x.cpu(), block, dtype, pow2)
    assert q.dtype == dtype and s.dtype == torch.float32
    assert q.shape == eq.shape and s.shape == es.shape
    assert torch.equal(s.cpu().double(), es)
    assert torch.equal(q.cpu().double(), eq)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("xtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 129), (127, 7), (130, 300), (257, 1024)])
def test_quantize(shape, block, xtype, dtype, pow2):
    x = rand(*shape, seed=shape[0] + shape[1]).mul(3).to(xtype).cuda()
    check_quantized(x, block, dtype, pow2, *sg.f8_quantize(x, block, dtype=dtype, pow2=pow2))


@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("shape", [(1, 5), (200, 333), (512, 256)])
def test_quantize_pair_is_both(shape, dtype):
    x = rand(*shape, seed=3).to(torch.bfloat16).cuda()
    q, s, qc, sc = sg.f8_quantize_pair(x, dtype=dtype)
    check_quantized(x, (1, 128), dtype, False, q, s)
    check_quantized(x, (128, 1), dtype, False, qc, sc)


@pytest.mark.parametrize("block", BLOCKS)
def test_quantize_many_rows(block):
    # enough blocks for several rounds of each block kernel
    x = rand(3000, 1500, seed=4).to(torch.bfloat16).cuda()
    check_quantized(x, block, E4, False, *sg.f8_quantize(x, block))


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_quantize_strided_and_unaligned(block, offset):
    buf = torch.full((140, 401), float("nan")).cuda()
    view = buf[2:135, offset:offset + 390]
    view.copy_(rand(133, 390, seed=5))
    check_quantized(view, block, E4, False, *sg.f8_quantize(view, block))


@pytest.mark.parametrize("block", BLOCKS)
def test_quantize_extremes(block):
    """Zero blocks, the smallest and the largest numbers, ties of the rounding."""
    x = torch.zeros(256, 256)
    x[0, :130] = 1e-45
    x[:, 140] = 3.0e38
    x[130:, 5] = torch.arange(126) * (448 / 126 / 16)
    x[130, 5] = 448.0
    check_quantized(x.cuda(), block, E4, False, *sg.f8_quantize(x.cuda(), block))
    check_quantized(x.cuda(), block, E4, True, *sg.f8_quantize(x.cuda(), block, pow2=True))
    t = torch.arange(-448, 448, 0.5).repeat(128, 1)[:, :1792]  # every tie above 8, scale 1
    t[:, ::128] = 448.0
    check_quantized(t.cuda(), block, E4, False, *sg.f8_quantize(t.cuda(), block))


@pytest.mark.parametrize("block", BLOCKS)
def test_quantize_not_finite(block):
    x = rand(256, 256, seed=6)
    x[3, 7], x[200, 201] = float("nan"), float("-inf")
    q, s = sg.f8_quantize(x.cuda(), block)
    q, s = q.cpu().float(), s.cpu()
    br, bc = block
    bi, bj = 3 // br, 7 // bc
    assert torch.isnan(s[bi, bj]) and torch.isnan(q[3, 7])
    bi, bj = 200 // br, 201 // bc
    assert torch.isinf(s[bi, bj]) and torch.isnan(q[200, 201])
    assert torch.isfinite(s).sum() == s.numel() - 2


@pytest.mark.parametrize("shape", [(0, 5), (5, 0), (0, 0)])
def test_quantize_empty(shape):
    q, s = sg.f8_quantize(torch.empty(shape, device="cuda"))
    assert q.shape == shape and s.shape == (shape[0], (shape[1] + 127) // 128)


def test_quantize_leaves_the_padding():
    x = rand(5, 100, seed=7).cuda()
    q = torch.full((5, 112), 0x5a, dtype=torch.uint8, device="cuda")
    s = torch.empty(5, 1, device="cuda")
    rc = sg.lib.f8_quantize(5, 100, x.data_ptr(), 0, 100, 1, 128, 0, 0, q.data_ptr(), 112,
                            s.data_ptr(), 1, 1, None, 0, None, 0, 0,
                            torch.cuda.current_stream().cuda_stream or None)
    assert rc == 0
    assert (q[:, 100:] == 0x5a).all()
    assert torch.equal(q[:, :100].view(E4).cpu().double(), plain.quantize(x.cpu(), (1, 128), E4, False)[0])


# ------------------------------------------------------------------------------ product

def operand(rows, cols, block, dtype, seed):
    """Random bytes of the format and random scales of any size: a quantised matrix that no
    quantiser made."""
    q = plain.round_to(rand(rows, cols, seed=seed).double() * 20, dtype).to(dtype)
    g = torch.Generator().manual_seed(seed + 1)
    br, bc = block
    s = torch.exp(torch.randn(-(-rows // br), -(-cols // bc), generator=g))
    return q, s


def on_gpu(q, pad=0):
    rows, cols = q.shape
    buf = torch.full((rows, (cols + 15) // 16 * 16 + pad), 0x7f, dtype=torch.uint8)  # NaN in E4M3
    buf[:, :cols] = q.view(torch.uint8)
    return buf.cuda().view(q.dtype)[:, :cols]


def check(M, N, K, transa, transb, ga, gb, da, db, dtype, alpha=1.0, beta=0.0, seed=0, pad=0):
    ablk = (ga, 128) if not transa else (128, ga)
    bblk = (128, gb) if not transb else (gb, 128)
    qa, sa = operand(*((K, M) if transa else (M, K)), ablk, da, seed + 1)
    qb, sb = operand(*((N, K) if transb else (K, N)), bblk, db, seed + 11)
    a, b = plain.values(qa, sa), plain.values(qb, sb)
    a, b = (a.t() if transa else a), (b.t() if transb else b)
    d0 = rand(M, N, seed=seed + 21, scale=100.0).to(dtype) if beta else None
    out = None
    if beta:
        wide = torch.full((M, N + 5), 7.0, dtype=dtype).cuda()
        out = wide[:, 2:2 + N]
        out.copy_(d0)
    got = sg.f8_matmul(on_gpu(qa, pad), sa.cuda(), on_gpu(qb, pad), sb.cuda(), transa=transa,
                       transb=transb, alpha=alpha, beta=beta, out=out, out_dtype=dtype)
    assert got.dtype == dtype and tuple(got.shape) == (M, N)
    R = alpha * (a @ b)
    S = abs(alpha) * (a.abs() @ b.abs())
    tol = (K + 8) * 2.0 ** -23 * S
    if beta:
        R = R + beta * d0.double()
        tol = tol + 2.0 ** -23 * abs(beta) * d0.double().abs()
        assert (wide[:, :2] == 7.0).all() and (wide[:, 2 + N:] == 7.0).all()
    tol = tol + ROUND[dtype] * R.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = (got.cpu().double() - R).abs()
    assert (err <= tol).all(), f"max err/tol {(err / tol).max().item():.3g}"


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 130, 300), (2, 1, 16), (7, 33, 65), (16, 256, 1024),
          (17, 129, 127), (64, 100, 257), (127, 255, 129), (128, 256, 512), (129, 257, 640),
          (300, 500, 200), (1, 2048, 4096), (1000, 70, 1500)]


@pytest.mark.parametrize("transa", [False, True])
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product_shapes(shape, transa, transb):
    check(*shape, transa, transb, 1, 128, E4, E4, torch.bfloat16)


@pytest.mark.parametrize("ga", [1, 128])
@pytest.mark.parametrize("gb", [1, 128])
@pytest.mark.parametrize("da", [E4, E5])
@pytest.mark.parametrize("db", [E4, E5])
@pytest.mark.parametrize("shape", [(20, 300, 333), (200, 140, 260), (1500, 1400, 130)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_scales_and_formats(shape, da, db, ga, gb):
    check(*shape, False, True, ga, gb, da, db, torch.float32)
    check(*shape, True, False, ga, gb, da, db, torch.float32, pad=16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(3, 260, 700), (150, 270, 200), (513, 300, 1000)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("alpha,beta", [(0.5, -2.0), (1e-2, 1.0)])
def test_product_alpha_beta(shape, dtype, alpha, beta):
    # (alpha keeps FP16 results in its range)
    check(*shape, False, True, 1, 128, E4, E4, dtype, alpha=alpha * 2.0 ** -8, beta=beta)


def test_product_every_tile_width():
    """Row counts on both sides of each tile width's range, wide enough for many tiles."""
    for M in (1, 15, 31, 33, 63, 65, 127, 129, 255, 257):
        check(M, 1000, 384, False, True, 1, 128, E4, E4, torch.float32, seed=M)


def test_product_many_tiles_per_cta():
    qa, sa = operand(4224, 256, (1, 128), E4, 1)
    qb, sb = operand(4352, 256, (128, 128), E4, 2)
    got = sg.f8_matmul(on_gpu(qa), sa.cuda(), on_gpu(qb), sb.cuda(), transb=True,
                       out_dtype=torch.float32)
    a, b = plain.values(qa, sa).cuda(), plain.values(qb, sb).cuda()
    err = (got.double() - a @ b.t()).abs()
    assert (err <= (256 + 16) * 2.0 ** -23 * (a.abs() @ b.abs().t())).all()


@pytest.mark.parametrize("transa", [False, True])
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("ga,gb", [(1, 128), (128, 128), (1, 1)])
@pytest.mark.parametrize("shape", [(2305, 4400, 260), (2433, 4353, 129)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_large_tiles(shape, transa, transb, ga, gb):
    """Enough tiles for the largest tile width, an odd number of 128-row blocks among them."""
    M, N, K = shape
    ablk = (ga, 128) if not transa else (128, ga)
    bblk = (128, gb) if not transb else (gb, 128)
    qa, sa = operand(*((K, M) if transa else (M, K)), ablk, E4, 1)
    qb, sb = operand(*((N, K) if transb else (K, N)), bblk, E5, 2)
    d0 = torch.randn(M, N, device="cuda")
    got = sg.f8_matmul(on_gpu(qa), sa.cuda(), on_gpu(qb), sb.cuda(), transa=transa, transb=transb,
                       beta=1.0, out=d0.clone())
    a, b = plain.values(qa, sa).cuda(), plain.values(qb, sb).cuda()
    a, b = (a.t() if transa else a), (b.t() if transb else b)
    R = a @ b + d0.double()
    tol = (K + 8) * 2.0 ** -23 * (a.abs() @ b.abs()) + 2.0 ** -23 * (d0.double().abs() + R.abs())
    assert ((got.double() - R).abs() <= tol).all()


def test_product_scales_in_any_layout():
    M, N, K = 70, 200, 500
    qa, sa = operand(M, K, (1, 128), E4, 1)
    qb, sb = operand(N, K, (128, 128), E4, 2)
    a, b = on_gpu(qa), on_gpu(qb)
    want = sg.f8_matmul(a, sa.cuda(), b, sb.cuda(), transb=True)
    wide = torch.full((2 * M, 9), float("nan")).cuda()
    wide[::2, 1:9:2] = sa.cuda()
    got = sg.f8_matmul(a, wide[::2, 1:9:2], b, sb.cuda().t().contiguous().t(), transb=True)
    assert torch.equal(got, want)


def test_product_empty_and_quick_returns():
    qa, sa = operand(40, 64, (1, 128), E4, 1)
    qb, sb = operand(50, 64, (128, 128), E4, 2)
    a, b, sa, sb = on_gpu(qa), on_gpu(qb), sa.cuda(), sb.cuda()
    assert sg.f8_matmul(a[:0], sa[:0], b, sb, transb=True).shape == (0, 50)
    assert sg.f8_matmul(a, sa, b[:0], sb[:0], transb=True).shape == (40, 0)
    # no products: beta D, and zeros without reading D
    none = sg.f8_matmul(a[:, :0], sa[:, :0], b[:, :0], sb[:, :0], transb=True)
    assert none.shape == (40, 50) and (none == 0).all()
    d = torch.full((40, 50), 3.0, device="cuda")
    sg.f8_matmul(a, sa * float("nan"), b, sb, transb=True, alpha=0.0, beta=2.0, out=d)
    assert (d == 6.0).all()
    d.fill_(float("nan"))
    sg.f8_matmul(a, sa, b, sb, transb=True, alpha=0.0, out=d)
    assert (d == 0.0).all()
    d.fill_(float("nan"))
    sg.f8_matmul(a, sa, b, sb, transb=True, out=d)
    assert torch.isfinite(d).all()


@pytest.mark.parametrize("M", [8, 200])
def test_product_not_finite_stays_where_it_belongs(M):
    N, K = 300, 400
    x, w = rand(M, K, seed=1), rand(N, K, seed=2)
    x[5, 140] = float("nan")
    w[10, 3] = float("inf")
    q, s = sg.f8_quantize(x.cuda())
    wq, ws = sg.f8_quantize(w.cuda(), (128, 128))
    d = sg.f8_matmul(q, s, wq, ws, transb=True).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[5] = True          # the row of the NaN
    bad[:, :128] = True    # the rows of W that share a scale with the infinity
    assert torch.equal(~torch.isfinite(d), bad)


@pytest.mark.parametrize("shape", [(1, 4096, 4096), (64, 512, 2048), (300, 300, 300)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_same_bits_every_time(shape):
    M, N, K = shape
    qa, sa = operand(M, K, (1, 128), E4, 1)
    qb, sb = operand(N, K, (128, 128), E4, 2)
    args = (on_gpu(qa), sa.cuda(), on_gpu(qb), sb.cuda())
    first = sg.f8_matmul(*args, transb=True, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(first, sg.f8_matmul(*args, transb=True, out_dtype=torch.float32))


@pytest.mark.parametrize("shape", [(1, 14336, 4096), (16, 4096, 8192)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_cold_weights_back_to_back(shape):
    """Weights from memory, not from the cache: copies of neighbouring k blocks land in any order."""
    M, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda")
    q, s = sg.f8_quantize(x)
    ws = [sg.f8_quantize(torch.randn(N, K, generator=g, device="cuda"), (128, 128))
          for _ in range(6)]
    first = [sg.f8_matmul(q, s, *w, transb=True) for w in ws]
    for w, f in zip(ws, first):
        R = (q.double() * s.double().repeat_interleave(128, 1)) @ (
            w[0].double() * w[1].double().repeat_interleave(128, 0).repeat_interleave(128, 1)).t()
        assert (f.double() - R).norm() <= 2.0 ** -8 * R.norm()
    for _ in range(30):
        got = [sg.f8_matmul(q, s, *w, transb=True) for w in ws]
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_chain_on_another_stream_and_in_a_graph():
    x = rand(24, 1024, seed=1).to(torch.bfloat16).cuda()
    w = rand(512, 1024, seed=2).cuda()

    def chain():
        wq, ws = sg.f8_quantize(w, (128, 128))
        q, s = sg.f8_quantize(x)
        return sg.f8_matmul(q, s, wq, ws, transb=True)

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
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got.float(), 2 * want.float())


def test_product_offsets_past_32_bits():
    """D and the operands past 2^32 elements: sampled rows against the plain form."""
    M, N, K = 66048, 65664, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn(M, K, generator=g, device="cuda").to(E4)
    b = torch.randn(N, K, generator=g, device="cuda").to(E4)
    sa, sb = torch.rand(M, 1, device="cuda") + 0.5, torch.rand(N // 128, 1, device="cuda") + 0.5
    d = sg.f8_matmul(a, sa, b, sb, transb=True)
    assert d.numel() > 1 << 32
    for r in (0, 1, M // 2, M - 1):
        want = (a[r].double() * sa[r].double()) @ (b.double() * sb.double().repeat_interleave(128, 0)).t()
        bound = (K + 8) * 2.0 ** -23 * 200 + 2.0 ** -8 * want.abs()
        assert ((d[r].double() - want).abs() <= bound).all()


def test_quantize_offsets_past_32_bits():
    rows, cols = 66048, 65664
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    x[-1] = torch.arange(cols, device="cuda").to(torch.bfloat16)
    for block in BLOCKS:
        q, s = sg.f8_quantize(x, block)
        if block[0] == 1:
            eq, es = plain.quantize(x[-1:].cpu(), block, E4, False)
        else:
            tail = rows // 128 * 128  # rows is a multiple of 128: the last full block
            eq, es = plain.quantize(x[tail - 128:].cpu(), block, E4, False)
        assert torch.equal(s[-1].cpu().double(), es[-1])
        assert torch.equal(q[-1].cpu().double(), eq[-1])
        del q, s


def test_python_refusals_on_the_gpu():
    q = torch.zeros(64, 160, dtype=torch.uint8, device="cuda").view(E4)
    s, w = torch.ones(64, 2, device="cuda"), torch.ones(1, 2, device="cuda")
    ok = sg.f8_matmul(q, s, q, w, transb=True)
    assert ok.shape == (64, 64) and ok.dtype == torch.bfloat16
    with pytest.raises(ValueError):  # one scale for each 128 of k
        sg.f8_matmul(q, s[:, :1], q, w, transb=True)
    with pytest.raises(ValueError):  # rows of scales
        sg.f8_matmul(q, s[:63], q, w, transb=True)
    with pytest.raises(TypeError):
        sg.f8_matmul(q, s.half(), q, w, transb=True)
    with pytest.raises(ValueError):  # inner sizes
        sg.f8_matmul(q, s, q, torch.ones(1, 2, device="cuda"))
    with pytest.raises(ValueError):  # beta without out
        sg.f8_matmul(q, s, q, w, transb=True, beta=1.0)
    with pytest.raises(ValueError):  # out's shape
        sg.f8_matmul(q, s, q, w, transb=True, out=torch.zeros(64, 65, device="cuda"))
    with pytest.raises(TypeError):  # out's type
        sg.f8_matmul(q, s, q, w, transb=True, out=torch.zeros(64, 64, device="cuda").double())
    with pytest.raises(ValueError):  # unit column stride
        sg.f8_matmul(q, s, q, w, transb=True, out=torch.zeros(64, 64, device="cuda").t()[::2].t())
    with pytest.raises(sg.SgemmError) as e:  # rows of 24 bytes: not what TMA can read
        t = torch.zeros(64, 24, dtype=torch.uint8, device="cuda").view(E4)
        sg.f8_matmul(t, torch.ones(64, 1, device="cuda"), t, torch.ones(1, 1, device="cuda"),
                     transb=True)
    assert e.value.status == -9


def test_overlapping_rows_are_refused():
    """A gradient that autograd expanded, and a sliding window: their rows share elements, so no
    leading dimension describes them."""
    y = torch.zeros(8, 256, device="cuda", requires_grad=True)
    seen = []
    y.register_hook(seen.append)
    (y.sum(0) * torch.arange(256, device="cuda")).sum().backward()
    dy = seen[0]
    assert dy.stride() == (0, 1)
    window = torch.zeros(400, device="cuda").unfold(0, 256, 1)
    for x in (dy, window):
        for call in (sg.f8_quantize, sg.f8_quantize_pair):
            with pytest.raises(ValueError, match="overlap"):
                call(x)
        q, s = sg.f8_quantize(x.contiguous())
        w, ws = sg.f8_quantize(x.contiguous(), (128, 128))
        rows = x.shape[0]
        for out in (dy[:, :rows] if rows == 8 else window[:, :rows],
                    torch.zeros(1, rows, device="cuda").expand(rows, rows)):
            with pytest.raises(ValueError, match="overlap"):
                sg.f8_matmul(q, s, w, ws, transb=True, out=out)
        with pytest.raises(ValueError, match="overlap"):
            sg.f8_matmul(q[:1].expand(rows, 256), s, w, ws, transb=True)


@pytest.mark.parametrize("power", [-126, -125, -118, -116, -112, -109, -101, -100, -99, -60])
@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("xtype", [torch.float32, torch.bfloat16])
def test_quantize_ties_at_small_scales(power, dtype, xtype):
    """Numbers next to the ties of the format's smallest numbers, under scales down to the least."""
    rows, cols = 128, 256
    g = torch.Generator().manual_seed(200 + power)
    least = 2.0 ** (-9 if dtype == E4 else -16)
    top = (1.0 + torch.rand(rows, cols // 128, generator=g)) * plain.LARGEST[dtype]
    top = torch.ldexp(top, torch.tensor(power)).to(xtype).float()
    s = (top.double() / plain.LARGEST[dtype]).float().repeat_interleave(128, 1)
    tie = (torch.randint(0, 16, (rows, cols), generator=g) + 0.5) * least
    x = (tie.double() * s.double()).float()
    near = torch.randint(-2, 3, (rows, cols), generator=g)
    x = (x.view(torch.int32) + near).clamp_min(0).int().view(torch.float32)
    x[:, ::128] = top
    x = (x * (1 - 2 * torch.randint(0, 2, (rows, cols), generator=g))).to(xtype)
    for y in (x, x.t().contiguous()):
        for block in BLOCKS:
            check_quantized(y.cuda(), block, dtype, False, *sg.f8_quantize(y.cuda(), block, dtype=dtype))
        check_quantized(y.cuda(), (128, 1), dtype, True,
                        *sg.f8_quantize(y.cuda(), (128, 1), dtype=dtype, pow2=True))
        q, s1, qc, sc = sg.f8_quantize_pair(y.cuda(), dtype=dtype)
        check_quantized(y.cuda(), (1, 128), dtype, False, q, s1)
        check_quantized(y.cuda(), (128, 1), dtype, False, qc, sc)


def test_quantize_small_beside_large_and_not_finite():
    """Columns and rows of every magnitude in one tile: each keeps to its own scale."""
    x = rand(256, 256, seed=31) * 2.0 ** torch.linspace(-140, 100, 256)[None, :]
    x[:, 7] = 0.0
    x[5, 9] = float("nan")
    x[6, 200] = float("-inf")
    for xtype in (torch.float32, torch.bfloat16):
        for y in (x.to(xtype), x.to(xtype).t().contiguous()):
            q, s, qc, sc = sg.f8_quantize_pair(y.cuda())
            for block, got, scale in (((1, 128), q, s), ((128, 1), qc, sc)):
                alone, salone = sg.f8_quantize(y.cuda(), block)
                assert torch.equal(got.view(torch.uint8), alone.view(torch.uint8))
                fine = torch.isfinite(y)
                keep = fine.view(-1, y.shape[0] // 2, y.shape[1]) if block[0] == 128 else \
                    fine.view(y.shape[0], -1, 128)
                keep = keep.all(dim=1 if block[0] == 128 else 2)  # blocks of finite numbers
                clean = torch.where(fine, y, torch.zeros_like(y))
                eq, es = plain.quantize(clean, block, E4, False)
                assert torch.equal(scale.cpu().double()[keep], es[keep])
                br, bc = block
                spread = keep[plain.block_index(256, br)][:, plain.block_index(256, bc)]
                assert torch.equal(got.cpu().double()[spread], eq[spread])
                assert not torch.isfinite(scale.cpu()[~keep]).any()
                assert torch.isnan(got.cpu().float()[~fine]).all()


@pytest.mark.parametrize("cols", [(1 << 31) - 64, (1 << 31) - 128])
def test_quantize_longest_row(cols):
    """A row whose number of columns rounded up to whole blocks passes 32 bits."""
    x = torch.full((1, cols), 2.0, dtype=torch.float16, device="cuda")
    x[0, -64:] = torch.arange(64, device="cuda")
    q, s = sg.f8_quantize(x)
    assert q.shape == (1, cols) and s.shape == (1, 1 << 24 if cols % 128 else (1 << 24) - 1)
    first = cols // 128 * 128 - (128 if cols % 128 == 0 else 0)
    for at, n in ((0, 256), (cols // 256 * 128, 256), (first, cols - first)):
        eq, es = plain.quantize(x[:, at:at + n].cpu(), (1, 128), E4, False)
        assert torch.equal(q[:, at:at + n].cpu().double(), eq)
        assert torch.equal(s[:, at // 128:(at + n + 127) // 128].cpu().double(), es)
    sample = torch.arange(0, s.shape[1] - 1, 997, device="cuda")
    assert (s[0, sample] == s[0, 0]).all()


def test_quantize_most_rows():
    """2^31 - 1 rows of one column: the last warp's lanes without a row have none to compute with."""
    rows, guard = (1 << 31) - 1, 256
    x = torch.full((rows,), 2.0, dtype=torch.float16, device="cuda")
    x[-4:] = torch.tensor([1.0, -3.0, 0.0, 5.0], device="cuda")
    q = torch.full((rows + 2 * guard,), 0x5a, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + 2 * guard,), 7.0, device="cuda")
    rc = sg.lib.f8_quantize(rows, 1, x.data_ptr(), 2, 1, 1, 128, 0, 0, q.data_ptr() + guard, 1,
                            s.data_ptr() + 4 * guard, 1, 1, None, 0, None, 0, 0,
                            torch.cuda.current_stream().cuda_stream or None)
    assert rc == 0
    eq, es = plain.quantize(x[-6:, None].cpu(), (1, 128), E4, False)
    assert torch.equal(q[-guard - 6:-guard].view(E4).cpu().double(), eq[:, 0])
    assert torch.equal(s[-guard - 6:-guard].cpu().double(), es[:, 0])
    assert (q[guard:-guard - 4].view(torch.int8) == 0x7e).all()  # 448
    assert (q[:guard] == 0x5a).all() and (q[-guard:] == 0x5a).all()
    assert (s[:guard] == 7.0).all() and (s[-guard:] == 7.0).all()


@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("ga,gb", [(1, 1), (1, 128), (128, 128)])
@pytest.mark.parametrize("powers", [(88, -100), (-100, 88), (-60, -66), (40, 48), (-126, 88)])
@pytest.mark.parametrize("shape", [(20, 300, 333), (330, 300, 260)], ids=lambda s: "x".join(map(str, s)))
def test_product_range_of_scales(shape, powers, ga, gb, dtype):
    """Scales at the ends of what the header allows, and a block of zeros under the least scale."""
    M, N, K = shape
    qa, sa = operand(M, K, (ga, 128), dtype, 1)
    qb, sb = operand(N, K, (gb, 128), dtype, 2)
    u = torch.rand(sa.shape, generator=torch.Generator().manual_seed(3))
    sa, sb = torch.ldexp(1 - u / 2 if powers[0] > 0 else 1 + u, torch.tensor(powers[0])), \
        torch.full_like(sb, 2.0 ** powers[1])
    qa[:ga, :128], sa[0, 0] = torch.zeros(min(ga, M), 128).to(dtype), 2.0 ** -126
    a, b = plain.values(qa, sa), plain.values(qb, sb)
    # (alpha keeps D in FP32's range)
    alpha = 2.0 ** -(sum(powers) // 2)
    d = sg.f8_matmul(on_gpu(qa), sa.cuda(), on_gpu(qb), sb.cuda(), transb=True, alpha=alpha,
                     out_dtype=torch.float32).cpu().double()
    R, S = alpha * (a @ b.t()), abs(alpha) * (a.abs() @ b.abs().t())
    assert ((d - R).abs() <= (K + 8) * 2.0 ** -23 * S + 2.0 ** -23 * R.abs()).all()
