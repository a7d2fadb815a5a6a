"""Workloads of what stands around a linear layer's products: layer norm in front of it and its
gradients, clipping of the gradients before the update, and the layer served in 8-bit integers.

`run` computes a case in elementary torch operations, in 32 bits where that holds what matters, or,
with `own` set, through the package's entry points (layer_norm, layer_norm_backward,
clip_grad_norm, i8_quantize, i8_linear). `exact` computes the same from the definitions in 64 bits.

Operators and their definitions:
  norm           mean, var over a row of x (var: the mean of squared distances from the mean);
                 r = 1 / sqrt(var + eps); y = (x - mean) r w + b
  norm-backward  h = (x - mean) r, g = dy w; dx = r (g - mean(g) - h mean(g h)) along a row;
                 dw = sum of dy h, db = sum of dy over the rows
  clip           norm = sqrt(sum of squares of all elements of all tensors);
                 out = g * min(1, max_norm / (norm + eps))
  quantise       for each row of x: a = max(max|x|, 2^-119); scale = a / 127; q = x (127 / a) rounded
                 to whole numbers, ties to even; both quotients in 32 bits, the product exact
  linear         out[i, j] = sx[i] sw[j] sum_k x[i, k] w[j, k] + bias[j] on 8-bit integers
"""
import math
import random

import torch

own = False

TYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
CLIP_EPS = 1e-6
LEAST = 2.0 ** -119


def listed():
    return [
        # one token in front of a serving product: launch latency
        dict(name="norm-token", op="norm", rows=1, cols=4096, type="bf16"),
        # a training step's activations, with the statistics that the backward pass takes
        dict(name="norm-activations", op="norm", rows=8192, cols=4096, type="bf16"),
        # their gradients, with those of the weight and the bias
        dict(name="norm-backward", op="norm-backward", rows=8192, cols=4096, type="bf16"),
        # odd and ragged, all in 32 bits
        dict(name="norm-backward-ragged", op="norm-backward", rows=4099, cols=777, type="f32"),
        # the gradients of two MLP layers, added up in 32 bits, clipped before the update
        dict(name="clip-layers", op="clip", layers=2, width=4096, inner=14336, type="f32",
             over=True, place=False),
        # biases, norms' weights and small matrices of two types: many tensors, little data
        dict(name="clip-many-small", op="clip", count=200, largest=65536, mix=1, type="mixed",
             over=True, place=False),
        # one token's activations in front of a serving product
        dict(name="quantize-token", op="quantize", rows=1, cols=4096, type="bf16"),
        # a prompt's activations
        dict(name="quantize-activations", op="quantize", rows=8192, cols=4096, type="bf16"),
        # serving, one token: the weight is read once
        dict(name="linear-token", op="linear", m=1, n=14336, k=4096, type="bf16", bias=False),
        # serving, a small batch of tokens
        dict(name="linear-16-tokens", op="linear", m=16, n=4096, k=8192, type="bf16", bias=True),
        # odd and ragged, a few hundred tokens
        dict(name="linear-ragged", op="linear", m=517, n=3001, k=777, type="f32", bias=True),
        # prompts: the largest product
        dict(name="linear-prompts", op="linear", m=8192, n=14336, k=4096, type="bf16",
             bias=False),
    ]


def _log_between(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _size(rng, low, high):
    """A size of the range: a multiple of 64 or any number, half and half."""
    v = _log_between(rng, low, high)
    return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["norm", "norm-backward", "clip", "quantize", "linear", "linear"])
    if op in ("norm", "norm-backward", "quantize"):
        rows = _size(rng, 1, 16384)
        return dict(op=op, rows=rows, cols=_size(rng, 16, min(16384, (1 << 25) // rows)),
                    type=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "clip":
        over = rng.random() < 0.7
        case = dict(op=op, type=rng.choice(["f32", "bf16", "mixed"]), over=over,
                    place=not over and rng.random() < 0.5)
        if rng.random() < 0.4:
            return dict(case, layers=rng.randint(1, 8), width=_size(rng, 64, 2048),
                        inner=_size(rng, 64, 4096))
        return dict(case, count=_log_between(rng, 1, 400), largest=_log_between(rng, 64, 1 << 20),
                    mix=rng.randint(0, 1 << 20))
    m, n, k = _size(rng, 1, 8192), _size(rng, 64, 14336), _size(rng, 64, 8192)
    return dict(op=op, m=m, n=n, k=max(64, min(k, (1 << 37) // (m * n))),
                type=rng.choice(["bf16", "bf16", "f16", "f32"]), bias=rng.random() < 0.5)


# ---------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Normal values on channels of different spread and mean, a few of them far larger."""
    spread = torch.exp(0.5 * _normal(g, 1, cols))
    spread = torch.where(torch.rand(1, cols, generator=g, device="cuda") < 0.01, 20 * spread,
                         spread)
    return (_normal(g, rows, cols) + 0.3 * _normal(g, 1, cols)) * spread


def _gradients(g, rows, cols):
    """Small normal values on tokens of different weight."""
    return 1e-5 * _normal(g, rows, cols) * torch.exp(_normal(g, rows, 1))


def _weights(g, rows, cols):
    return _normal(g, rows, cols) / math.sqrt(cols)


def _sizes(case):
    """Elements of each gradient of a clip case."""
    if "layers" in case:
        w, i = case["width"], case["inner"]
        return case["layers"] * [w * i, i * w, i, w, w, w]
    r = random.Random(case["mix"])
    return [_log_between(r, 1, case["largest"]) for _ in range(case["count"])]


def _kinds(case):
    """Type of each gradient: that of the case, or 32 bits for one in three and bf16 for the others."""
    n = len(_sizes(case))
    if case["type"] == "mixed":
        return ["f32" if i % 3 == 0 else "bf16" for i in range(n)]
    return [case["type"]] * n


def _held(case, kind):
    """Where the tensors of one type begin in the buffer that holds them, and its elements."""
    at, starts = 0, []
    for size, k in zip(_sizes(case), _kinds(case)):
        starts.append(at)
        at += (size + 63) // 64 * 64 if k == kind else 0
    return starts, at


def _views(case, buffers):
    """The tensors of a clip case in the buffers that hold them."""
    starts = {kind: _held(case, kind)[0] for kind in buffers}
    return [buffers[kind][starts[kind][i]:starts[kind][i] + size]
            for i, (size, kind) in enumerate(zip(_sizes(case), _kinds(case)))]


def _prepare_clip(case, g):
    """Gradients of different magnitude, kept in one buffer for each type."""
    kinds = sorted(set(_kinds(case)))
    buffers = {k: torch.zeros(_held(case, k)[1], dtype=TYPE[k], device="cuda") for k in kinds}
    grads = _views(case, buffers)
    for v in grads:
        v.copy_(1e-3 * torch.exp(0.5 * _normal(g, 1)) * _normal(g, v.numel()))
    state = dict(case=case, grads=grads, buffers=buffers,
                 max_norm=(0.3e-3 if case["over"] else 1e-2) * math.sqrt(sum(_sizes(case))))
    if not case["place"]:
        state["out_buffers"] = {k: torch.zeros_like(b) for k, b in buffers.items()}
        state["out"] = _views(case, state["out_buffers"])
    return state


def _stored(q):
    """q in rows of a multiple of 16 bytes, as the package allocates it."""
    rows, cols = q.shape
    held = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=q.device)
    held[:, :cols] = q
    return held[:, :cols]


def _quantized(x):
    q, scale = _plain_quantize(x)
    return _stored(q), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "clip":
        return _prepare_clip(case, g)
    if case["op"] == "linear":
        x, sx = _quantized(_activations(g, case["m"], case["k"]))
        w, sw = _quantized(_weights(g, case["n"], case["k"]))
        return dict(case=case, x=x, sx=sx, w=w, sw=sw,
                    bias=_normal(g, case["n"]) if case["bias"] else None)
    x = _activations(g, case["rows"], case["cols"]).to(TYPE[case["type"]])
    state = dict(case=case, x=x)
    if case["op"] != "quantize":
        state["weight"] = 1 + 0.1 * _normal(g, case["cols"])
        state["bias"] = 0.1 * _normal(g, case["cols"])
    if case["op"] == "norm-backward":
        state["dy"] = _gradients(g, case["rows"], case["cols"]).to(TYPE[case["type"]])
        state["mean"], state["rstd"] = _statistics(x.float())
    return state


# ---------------------------------------------------------------------------- plain forms

def _statistics(x):
    mean = x.mean(dim=1)
    var = (x - mean[:, None]).square().mean(dim=1)
    return mean, 1.0 / torch.sqrt(var + EPS)


def _plain_norm(x, weight, bias):
    v = x.float()
    mean, rstd = _statistics(v)
    y = (v - mean[:, None]) * rstd[:, None] * weight + bias
    return y.to(x.dtype), mean, rstd


def _plain_norm_backward(dy, x, weight, mean, rstd):
    d = dy.float()
    h = (x.float() - mean[:, None]) * rstd[:, None]
    g = d * weight
    dx = rstd[:, None] * (g - g.mean(dim=1, keepdim=True) - h * (g * h).mean(dim=1, keepdim=True))
    return dx.to(x.dtype), (d * h).sum(dim=0), d.sum(dim=0)


def _plain_clip(grads, max_norm, out):
    # (sums of squares in 64 bits: they are long)
    total = torch.stack([v.float().square().sum(dtype=torch.float64) for v in grads]).sum()
    norm = total.sqrt()
    factor = (max_norm / (norm + CLIP_EPS)).clamp(max=1.0).float()
    [o.copy_(v.float() * factor) for v, o in zip(grads, out)]
    return norm.float()


def _plain_quantize(x):
    v = x.float()
    a = v.abs().amax(dim=1).clamp_min(LEAST)
    # (a division by a tensor: torch divides by a number with its reciprocal)
    top = torch.full_like(a, 127.0)
    # (the product in 64 bits, where it is exact: next to a border)
    q = torch.round(v.double() * (top / a).double()[:, None])
    return q.to(torch.int8), a / top


def _plain_linear(x, sx, w, sw, bias, dtype):
    y = (x.float() @ w.float().t()) * sx[:, None] * sw
    return (y if bias is None else y + bias).to(dtype)


# ---------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "norm":
        return _plain_norm(state["x"], state["weight"], state["bias"])
    if case["op"] == "norm-backward":
        return _plain_norm_backward(state["dy"], state["x"], state["weight"], state["mean"],
                                    state["rstd"])
    if case["op"] == "clip":
        norm = _plain_clip(state["grads"], state["max_norm"], state.get("out", state["grads"]))
        return dict(state.get("out_buffers", state["buffers"]), norm=norm)
    if case["op"] == "quantize":
        return _plain_quantize(state["x"])
    return _plain_linear(state["x"], state["sx"], state["w"], state["sw"], state["bias"],
                         TYPE[case["type"]])


def _run_own(case, state):
    import dense_fp32_matrix_08_gb300 as sg
    if case["op"] == "norm":
        return sg.layer_norm(state["x"], state["weight"], state["bias"], eps=EPS, stats=True)
    if case["op"] == "norm-backward":
        return sg.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"],
                                      state["weight"])
    if case["op"] == "clip":
        norm = sg.clip_grad_norm(state["grads"], state["max_norm"], eps=CLIP_EPS,
                                 out=state.get("out"))
        return dict(state.get("out_buffers", state["buffers"]), norm=norm)
    if case["op"] == "quantize":
        return sg.i8_quantize(state["x"])
    return sg.i8_linear(state["x"], state["sx"], state["w"], state["sw"], state["bias"],
                        out_dtype=TYPE[case["type"]])


# ---------------------------------------------------------------------------- least work

def work(case):
    if case["op"] == "clip":
        read = sum(s * SIZE[k] for s, k in zip(_sizes(case), _kinds(case)))
        return {"bytes": read * (1 if case["place"] else 2), "flops": 3 * sum(_sizes(case))}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n * (2 if case["bias"] else 1))
                + m * n * SIZE[case["type"]], "flops": 2 * m * n * k}
    r, c = case["rows"], case["cols"]
    held = r * c * SIZE[case["type"]]
    if case["op"] == "quantize":
        return {"bytes": held + r * c + 4 * r, "flops": 2 * r * c}
    if case["op"] == "norm":
        return {"bytes": 2 * held + 8 * (r + c), "flops": 7 * r * c}
    return {"bytes": 3 * held + 8 * r + 12 * c, "flops": 14 * r * c}


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "clip":
        flat = {k: b.double() for k, b in state["buffers"].items()}  # (zeros between tensors)
        norm = math.sqrt(sum(torch.dot(b, b).item() for b in flat.values()))
        factor = min(1.0, state["max_norm"] / (norm + CLIP_EPS))
        return dict({k: b.mul_(factor) for k, b in flat.items()},
                    norm=torch.tensor(norm, dtype=torch.float64))
    if case["op"] == "linear":
        total = torch.mm(state["x"].double(), state["w"].double().mT)  # (whole numbers: exact)
        y = torch.outer(state["sx"].double(), state["sw"].double()) * total
        return y if state["bias"] is None else y + state["bias"].double()
    x = state["x"].double()
    if case["op"] == "quantize":
        a = torch.maximum(x.abs().amax(1), torch.full_like(x[:, 0], LEAST))
        # quotients rounded to 32 bits: from 53 they round as from the real number
        factor = (127.0 / a).float().double()
        return torch.round(factor[:, None] * x).to(torch.int8), a / 127.0
    weight = state["weight"].double()
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        y = torch.addcmul(state["bias"].double(), (x - mean[:, None]) * rstd[:, None], weight)
        return y, mean, rstd
    dy, r = state["dy"].double(), state["rstd"].double()[:, None]
    h = r * (x - state["mean"].double()[:, None])
    n = x.shape[1]
    g = weight * dy
    along = torch.einsum("ij,ij->i", g, h) / n
    dx = r * (g - g.sum(1, keepdim=True) / n - along[:, None] * h)
    return dx, torch.einsum("ij,ij->j", dy, h), dy.sum(0)
