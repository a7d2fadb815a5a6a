"""GPU tests of the `stream` argument of the operators that allocate their results: the results, and
that memory one stream still uses is not handed to another."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

ROWS, COLS = 1536, 1280


def rand(*shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def quantize(stream):
    x = rand(ROWS, COLS, seed=1)
    return (x,), lambda: sg.f8_quantize(x, (128, 128), stream=stream)


def quantize_pair(stream):
    x = rand(ROWS, COLS, seed=2, dtype=torch.bfloat16)
    return (x,), lambda: sg.f8_quantize_pair(x, stream=stream)


def matmul(stream):
    a = sg.f8_quantize(rand(ROWS, COLS, seed=3))
    b = sg.f8_quantize(rand(ROWS, COLS, seed=4), (128, 128))
    return (*a, *b), lambda: sg.f8_matmul(*a, *b, transb=True, stream=stream)


def matmul_into(stream):
    a = sg.f8_quantize(rand(ROWS, COLS, seed=3))
    b = sg.f8_quantize(rand(ROWS, COLS, seed=4), (128, 128))
    d = torch.ones(ROWS, ROWS, device="cuda")
    return (*a, *b, d), lambda: sg.f8_matmul(*a, *b, transb=True, beta=0.5, out=d, stream=stream)


def orthogonalize(stream):
    g = rand(300, COLS, seed=5)
    return (g,), lambda: sg.orthogonalize(g, steps=2, stream=stream)


CALLS = [quantize, quantize_pair, matmul, matmul_into, orthogonalize]


def several(result):
    return result if isinstance(result, tuple) else (result,)


def as_bytes(t):
    return t.contiguous().view(torch.uint8)


def behind(stream):
    """Work that keeps `stream` busy for some tens of milliseconds."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)


@pytest.mark.parametrize("how", ["stream", "handle", "current", "default"])
@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_results(make, how):
    want = [as_bytes(t).clone() for t in several(make(None)[1]())]
    side = torch.cuda.Stream()
    stream = {"stream": side, "handle": side.cuda_stream, "current": torch.cuda.current_stream(),
              "default": 0}[how]
    _, call = make(stream)
    side.wait_stream(torch.cuda.current_stream())
    got = several(call())
    torch.cuda.synchronize()
    assert all(torch.equal(as_bytes(g), w) for g, w in zip(got, want))


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_dropped_results_are_not_handed_on(make):
    """The caller drops a result while its stream has not written it yet, and allocates again."""
    side = torch.cuda.Stream()
    keep, call = make(side)
    behind(side)
    result = several(call())
    taken = {t.data_ptr(): t.untyped_storage().nbytes() for t in result}
    del result
    new = [torch.full((n,), 7, dtype=torch.uint8, device="cuda")
           for n in taken.values() for _ in range(4)]
    if make is not matmul_into:  # (there the result is the caller's)
        assert not taken.keys() & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in new)


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_dropped_inputs_are_not_handed_on(make):
    """The caller drops the inputs while the stream has not read them yet, and allocates again."""
    want = [as_bytes(t).clone() for t in several(make(None)[1]())]
    side = torch.cuda.Stream()
    inputs, call = make(side)
    behind(side)
    got = several(call())
    sizes = [t.untyped_storage().nbytes() for t in inputs]
    del inputs, call
    new = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(as_bytes(g), w) for g, w in zip(got, want))
    assert all((t == 7).all() for t in new)
