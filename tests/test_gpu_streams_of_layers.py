"""GPU tests of the `stream` argument of layer norm and its gradients, of clipping and of the linear layer on
8-bit integers, as test_gpu_streams has them for the other operators; and of calls from several threads on
streams of their own."""
import threading

import pytest
import torch

from test_gpu_streams import behind, rand, several

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_fp32_matrix_08_gb300 as sg

ROWS, COLS = 1536, 1280


def as_bytes(t):
    return t.reshape(-1).view(torch.uint8)


def norm(stream):
    x, w, b = rand(ROWS, COLS, seed=1, dtype=torch.bfloat16), rand(COLS, seed=2), rand(COLS, seed=3)
    return (x, w, b), lambda: sg.layer_norm(x, w, b, stats=True, stream=stream)


def norm_backward(stream):
    x, dy, w = rand(ROWS, COLS, seed=1), rand(ROWS, COLS, seed=2), rand(COLS, seed=3)
    mean, rstd = x.mean(1), 1 / x.std(1)
    return (x, dy, w, mean, rstd), lambda: sg.layer_norm_backward(dy, x, mean, rstd, w, stream=stream)


def norm_backward_alone(stream):
    x, dy = rand(ROWS, COLS, seed=1), rand(ROWS, COLS, seed=2)
    mean, rstd = x.mean(1), 1 / x.std(1)
    return (x, dy, mean, rstd), lambda: sg.layer_norm_backward(dy, x, mean, rstd, stream=stream)[0]


def clip(stream):
    grads = [rand(ROWS, COLS, seed=4), rand(77, seed=5, dtype=torch.float16)]
    out = [torch.zeros_like(g) for g in grads]
    return grads, lambda: (sg.clip_grad_norm(grads, 1.0, out=out, stream=stream), *out)


def quantize(stream):
    x = rand(ROWS, COLS, seed=6, dtype=torch.bfloat16)
    return (x,), lambda: sg.i8_quantize(x, stream=stream)


def linear(rows):
    def make(stream):
        x, w, b = sg.i8_quantize(rand(rows, COLS, seed=7)), sg.i8_quantize(rand(ROWS, COLS, seed=8)), rand(ROWS, seed=9)
        return (*x, *w, b), lambda: sg.i8_linear(*x, *w, b, stream=stream)
    make.__name__ = f"linear_{rows}"
    return make


OWN = [norm, norm_backward, norm_backward_alone, quantize, linear(1), linear(40), linear(700)]  # all results new
CALLS = OWN + [clip]


@pytest.mark.parametrize("how", ["stream", "handle", "current", "default"])
@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_results(make, how):
    want = [as_bytes(t).clone() for t in several(make(None)[1]())]
    side = torch.cuda.Stream()
    stream = {"stream": side, "handle": side.cuda_stream, "current": torch.cuda.current_stream(), "default": 0}[how]
    _, call = make(stream)
    side.wait_stream(torch.cuda.current_stream())
    got = several(call())
    torch.cuda.synchronize()
    assert all(torch.equal(as_bytes(g), w) for g, w in zip(got, want))


@pytest.mark.parametrize("make", OWN, ids=lambda f: f.__name__)
def test_dropped_results_are_not_handed_on(make):
    """The caller drops a result while its stream has not written it yet, and allocates again."""
    side = torch.cuda.Stream()
    keep, call = make(side)
    behind(side)
    result = several(call())
    taken = {t.data_ptr(): t.untyped_storage().nbytes() for t in result}
    del result
    new = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in taken.values() for _ in range(4)]
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


def test_several_threads_and_streams():
    """Calls of all operators at once: workspaces and tables are each call's own."""
    wants = [[as_bytes(t).clone() for t in several(make(None)[1]())] for make in CALLS]
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for turn in range(6):
                k = (i + turn) % len(CALLS)
                got = several(CALLS[k](None)[1]())
                stream.synchronize()
                if not all(torch.equal(as_bytes(g), w) for g, w in zip(got, wants[k])):
                    wrong.append((i, CALLS[k].__name__))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_graphs_that_share_the_pool():
    """Two captured graphs, replayed in turn and then at the same time on two streams."""
    graphs = []
    for make in (norm_backward, linear(700), clip):
        for _ in range(2):
            keep, call = make(None)
            want = [t.clone() for t in several(call())]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = several(call())
            graphs.append((graph, got, want, keep, call))
    for graph, got, *_ in graphs:
        for t in got:
            t.zero_()
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for turn in range(3):
        for (graph, *_), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, got, want, *_ in graphs:
            assert all(torch.equal(g, w) for g, w in zip(got, want))
