"""GPU tests of every plan of the 8-bit product and of the orthogonalisation (the shapes of plans.py),
against the definitions in 64 bits. Bounds as in test_gpu_f8.py and test_gpu_orthogonalize.py."""
import pytest
import torch

from plans import ORTHOGONALIZATIONS, PRODUCTS

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
ROUND = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(autouse=True)
def status_clear():
    yield
    assert sg.f8_gemm_status() == (0, 0) and sg.ns_orthogonalize_status() == (0, 0)


def operand(g, rows, cols, block, dtype):
    """(q, scales, values in 64 bits) of a quantised matrix; NaN bytes in the rows' padding."""
    br, bc = block
    held = torch.full((rows, (cols + 15) // 16 * 16), 0x7f, dtype=torch.uint8, device="cuda")
    q = (torch.randn(rows, cols, generator=g, device="cuda") * 20).to(dtype)
    held[:, :cols] = q.view(torch.uint8)
    s = torch.exp(torch.randn(-(-rows // br), -(-cols // bc), generator=g, device="cuda"))
    spread = s.double().repeat_interleave(br, 0)[:rows].repeat_interleave(bc, 1)[:, :cols]
    return held.view(dtype)[:, :cols], s, q.double() * spread


def product(shape, dtype, alpha, beta, pad, seed):
    """One product into columns `pad` .. of a wider matrix of sevens."""
    M, N, K, ta, tb, ar, bc = shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    qa, sa, a = operand(g, K, M, (128, ar), E5) if ta else operand(g, M, K, (ar, 128), E5)
    qb, sb, b = operand(g, N, K, (bc, 128), E4) if tb else operand(g, K, N, (128, bc), E4)
    a, b = a.t() if ta else a, b.t() if tb else b
    wide = torch.full((M, (N + 15) // 8 * 8 + pad), 7.0, dtype=dtype, device="cuda")
    out = wide[:, pad:pad + N]
    d0 = (50 * torch.randn(M, N, generator=g, device="cuda")).to(dtype)
    out.copy_(d0 if beta else torch.full_like(d0, float("nan")))
    assert sg.f8_matmul(qa, sa, qb, sb, transa=bool(ta), transb=bool(tb), alpha=alpha, beta=beta,
                        out=out) is out
    R, tol = alpha * (a @ b), (K + 8) * 2.0 ** -23 * abs(alpha) * (a.abs() @ b.abs())
    if beta:
        R += beta * d0.double()
        tol += 2.0 ** -23 * abs(beta) * d0.double().abs()
    tol += ROUND[dtype] * R.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = (out.double() - R).abs()
    assert (err <= tol).all(), f"{shape}: max err/tol {(err / tol).max().item():.3g}"
    assert (wide[:, :pad] == 7.0).all() and (wide[:, pad + N:] == 7.0).all()


@pytest.mark.parametrize("key", PRODUCTS, ids=lambda k: "-".join(map(str, k)))
def test_products(key):
    for i, shape in enumerate(PRODUCTS[key]):
        M, N, K, ta, tb, ar, bc = shape
        p = sg.f8_gemm_plan(M, N, K, transa=ta, transb=tb, a_rows=ar, b_cols=bc)
        assert (int(p["exchanged"]), p["tile_cols"], p["split"]) == key
        product(shape, torch.float32, 1.0, 0.0, 0, i)
        product(shape, torch.float32, -0.5, 0.75, 3, i)
        product(shape, torch.bfloat16, 1.0, 0.0, 8, i)
        product(shape, torch.bfloat16, 0.5, -2.0, 1, i)
        product(shape, torch.float16, 2.0 ** -9, 0.0, 5, i)


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("key", ORTHOGONALIZATIONS, ids=lambda k: "-".join(map(str, k)))
def test_orthogonalizations(key, tall):
    batch, m, n = ORTHOGONALIZATIONS[key]
    rows, cols = (n, m) if tall else (m, n)
    p = sg.ns_orthogonalize_plan(batch, rows, cols)
    assert (p["tile_cols"], "".join("-" if s == 1 else "a" if w == 0 else "r"
                                    for s, w in zip(p["split"], p["whole"]))) == key
    gen = torch.Generator(device="cuda").manual_seed(batch + m + n)
    g = torch.randn(batch, rows, cols, generator=gen, device="cuda")
    a, b, c = 3.4445, -4.7750, 2.0315
    x = g.double().mT if tall else g.double()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + 1e-7)
    for _ in range(5):
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    x = x.mT if tall else x
    bound = 2.0 ** -20 * sum(4.0 ** k for k in range(5))
    norm = x.square().sum(dim=(1, 2)).sqrt()
    got = sg.orthogonalize(g)
    err = (got.double() - x).square().sum(dim=(1, 2)).sqrt()
    assert (err <= (bound + ROUND[torch.float32]) * norm).all(), (err / norm).max()
    # into a wider matrix, in 16 bits and with the old values
    for dtype, pad in ((torch.bfloat16, 3), (torch.float16, 8), (torch.float32, 1)):
        wide = torch.full((batch, rows, (cols + 15) // 8 * 8 + pad), 7.0, dtype=dtype, device="cuda")
        out = wide[:, :, pad:pad + cols]
        w = torch.randn(batch, rows, cols, generator=gen, device="cuda").to(dtype)
        out.copy_(w)
        sg.orthogonalize(g, alpha=-0.5, beta=0.25, out=out)
        want = 0.25 * w.double() - 0.5 * x
        err = (out.double() - want).square().sum(dim=(1, 2)).sqrt()
        tol = 0.5 * (bound + ROUND[torch.float32]) * norm + \
            ROUND[dtype] * want.square().sum(dim=(1, 2)).sqrt()
        assert (err <= tol).all(), (err / tol).max()
        assert (wide[:, :, :pad] == 7.0).all() and (wide[:, :, pad + cols:] == 7.0).all()
