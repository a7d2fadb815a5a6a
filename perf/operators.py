"""Workloads of the 8-bit block-scaled product, its quantiser and the Newton-Schulz
orthogonalisation: what a linear layer's training step and its serving call ask of them.

`run` computes a case in elementary 32-bit torch operations, or, with `own` set, through the
package's entry points (f8_quantize, f8_quantize_pair, f8_matmul, orthogonalize). `exact`
computes the same from the definitions in 64 bits.

Operators and their definitions:
  quantise   for each block b of x (1 x 128, 128 x 1 or 128 x 128 elements):
             s_b = max(max|x| / F, 2^-126), F the format's largest number (448 for e4m3,
             57344 for e5m2), with pow2 the least power of two not below that;
             q = x / s_b rounded to the format (nearest, ties to even)
  product    D = op(A) op(B) + beta D, op(A)[i, k] = qA sA with one scale for each 128 of k
             and each row (or 128 rows), op(B) alike; D in bf16 or fp32
  orthogonalise  X = G / (|G|_F + eps), then `steps` times X <- (a I + b S + c S^2) X with
             S = X X^T taken on the shorter side
"""
import math

import torch

own = False

BLOCK = 128
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
FORMAT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # one token's activations in front of a serving product: launch latency
        dict(name="quantize-token", op="quantize", rows=1, cols=4096, type="bf16", block="row",
             format="e4m3", pow2=False),
        # activations of a training step: rows for the forward product, columns for the weight
        # gradient, from one read
        dict(name="quantize-activations-pair", op="quantize", rows=8192, cols=4096, type="bf16",
             block="pair", format="e4m3", pow2=False),
        # a master weight after its update
        dict(name="quantize-weight", op="quantize", rows=14336, cols=4096, type="f32",
             block="square", format="e4m3", pow2=False),
        # serving, one token: the weight is read once
        dict(name="product-token", op="product", kind="forward", m=1, n=4096, k=4096,
             type="bf16", format="e4m3", pow2=False),
        # serving, a small batch of tokens
        dict(name="product-16-tokens", op="product", kind="forward", m=16, n=4096, k=8192,
             type="bf16", format="e4m3", pow2=False),
        # training, forward: the largest product
        dict(name="product-forward", op="product", kind="forward", m=8192, n=14336, k=4096,
             type="bf16", format="e4m3", pow2=False),
        # training, input gradient, odd and ragged, gradients in the wide-range format
        dict(name="product-input-gradient-ragged", op="product", kind="dgrad", m=4099, n=3001,
             k=777, type="bf16", format="e5m2", pow2=False),
        # training, weight gradient added to a 32-bit accumulator
        dict(name="product-weight-gradient", op="product", kind="wgrad", m=4096, n=4096, k=8192,
             type="f32", format="e4m3", pow2=False),
        # the update of one small matrix: latency of a chain of small products
        dict(name="orthogonalize-256", op="orthogonalize", batch=1, m=256, n=256, type="f32",
             steps=5),
        # several equal matrices at once (one for each layer or expert)
        dict(name="orthogonalize-8x1024", op="orthogonalize", batch=8, m=1024, n=1024,
             type="bf16", steps=5),
        # a tall, odd-sized matrix
        dict(name="orthogonalize-tall-ragged", op="orthogonalize", batch=1, m=4097, n=777,
             type="bf16", steps=5),
        # a large weight's update in full precision
        dict(name="orthogonalize-4096", op="orthogonalize", batch=1, m=4096, n=4096, type="f32",
             steps=5),
    ]


def _log_between(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _size(rng, low, high):
    """A size of the range: a multiple of 64 or any number, half and half."""
    v = _log_between(rng, low, high)
    return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "orthogonalize"])
    if op == "quantize":
        rows = _size(rng, 1, 16384)
        return dict(op=op, rows=rows, cols=_size(rng, 16, min(14336, (1 << 26) // rows)),
                    type=rng.choice(["f32", "bf16", "f16"]),
                    block=rng.choice(["row", "column", "square", "pair"]),
                    format=rng.choice(["e4m3", "e4m3", "e5m2"]), pow2=rng.random() < 0.3)
    if op == "product":
        kind = rng.choice(["forward", "forward", "dgrad", "wgrad"])
        m = _size(rng, 1 if kind == "forward" else 64, 8192)
        n, k = _size(rng, 64, 14336), _size(rng, 64, 8192)
        k = max(64, min(k, (1 << 38) // (m * n)))
        return dict(op=op, kind=kind, m=m, n=n, k=k, type="f32" if kind == "wgrad" else "bf16",
                    format=rng.choice(["e4m3", "e5m2"]) if kind != "forward" else "e4m3",
                    pow2=rng.random() < 0.3)
    m, n = _size(rng, 16, 4096), _size(rng, 16, 4096)
    batch = rng.choice([1, 1, 2, 3, 8])
    while batch > 1 and batch * m * n * min(m, n) > 1 << 33:
        batch -= 1
    return dict(op=op, batch=batch, m=m, n=n, type=rng.choice(["f32", "bf16"]),
                steps=rng.choice([5, 5, 6]))


# ---------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Normal values on channels of different spread, a few of them far larger."""
    spread = torch.exp(0.5 * _normal(g, 1, cols))
    spread = torch.where(torch.rand(1, cols, generator=g, device="cuda") < 0.01, 20 * spread,
                         spread)
    return _normal(g, rows, cols) * spread


def _gradients(g, rows, cols):
    """Small normal values on tokens of different weight."""
    return 1e-5 * _normal(g, rows, cols) * torch.exp(_normal(g, rows, 1))


def _weights(g, rows, cols):
    return _normal(g, rows, cols) / math.sqrt(cols)


def _momentum(g, batch, m, n):
    """A momentum matrix: a few strong directions over a broad bulk."""
    r = max(1, min(m, n) // 16)
    strength = torch.arange(1, r + 1, device="cuda", dtype=torch.float32) ** -0.5
    strong = (_normal(g, batch, m, r) * strength) @ _normal(g, batch, r, n)
    return 1e-3 * (_normal(g, batch, m, n) + strong)


def _stored(q):
    """q in rows of a multiple of 16 bytes, as the package allocates it."""
    rows, cols = q.shape
    held = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.uint8, device=q.device)
    held[:, :cols] = q.view(torch.uint8)
    return held.view(q.dtype)[:, :cols]


def _quantized(x, block, fmt, pow2):
    q, s = _plain_quantize(x, block, fmt, pow2)
    return _stored(q), s


def _operands(case, seed):
    """(qA, sA, blocks of A, transa, qB, sB, blocks of B, transb) of D = op(A) op(B)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, n, k, fmt, p2 = case["m"], case["n"], case["k"], case["format"], case["pow2"]
    if case["kind"] == "forward":  # y = x W^T: x is m x k, W is n x k
        a = _quantized(_activations(g, m, k), "row", "e4m3", p2) + ("row", False)
        b = _quantized(_weights(g, n, k), "square", "e4m3", p2) + ("square", True)
    elif case["kind"] == "dgrad":  # dx = dy W: dy is m x k, W is k x n
        a = _quantized(_gradients(g, m, k), "row", fmt, p2) + ("row", False)
        b = _quantized(_weights(g, k, n), "square", "e4m3", p2) + ("square", False)
    else:  # dW = dy^T x over k tokens: dy is k x m, x is k x n
        a = _quantized(_gradients(g, k, m), "column", fmt, p2) + ("column", True)
        b = _quantized(_activations(g, k, n), "column", "e4m3", p2) + ("column", False)
    return a + b


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "quantize":
        make = _weights if case["block"] == "square" else _activations
        return dict(case=case, x=make(g, case["rows"], case["cols"]).to(TYPE[case["type"]]))
    if case["op"] == "orthogonalize":
        x = _momentum(g, case["batch"], case["m"], case["n"])
        return dict(case=case, g=x.to(TYPE[case["type"]]))
    state = dict(case=case, operands=_operands(case, seed))
    if case["kind"] == "wgrad":  # the gradient accumulated so far
        state["d"] = 1e-4 * _normal(g, case["m"], case["n"])
    return state


# ---------------------------------------------------------------------------- plain forms

def _spread(s, shape, block):
    """Block scales as one for each element."""
    if block != "column":
        s = s.repeat_interleave(BLOCK, dim=1)[:, :shape[1]]
    if block != "row":
        s = s.repeat_interleave(BLOCK, dim=0)[:shape[0]]
    return s


def _plain_quantize(x, block, fmt, pow2):
    x = x.float()
    rows, cols = x.shape
    br = 1 if block == "row" else BLOCK
    bc = 1 if block == "column" else BLOCK
    nr, nc = -(-rows // br), -(-cols // bc)
    y = torch.zeros(nr * br, nc * bc, device=x.device)
    y[:rows, :cols] = x
    top = y.view(nr, br, nc, bc).abs().amax(dim=(1, 3))
    # (a division by a tensor: torch divides by a number with its reciprocal)
    s = (top / torch.full_like(top, LARGEST[fmt])).clamp_min(2.0 ** -126)
    if pow2:
        part, power = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), power - (part == 0.5).int())
    q = (x / _spread(s, x.shape, block)).clamp(-LARGEST[fmt], LARGEST[fmt]).to(FORMAT[fmt])
    if block == "row":
        s = s.t().contiguous().t()
    return q, s


def _plain_product(case, operands, d):
    qa, sa, ba, ta, qb, sb, bb, tb = operands
    a, b = qa.float() * _spread(sa, qa.shape, ba), qb.float() * _spread(sb, qb.shape, bb)
    y = (a.t() if ta else a) @ (b.t() if tb else b)
    if d is not None:
        return d.add_(y)
    return y.to(TYPE[case["type"]])


def _plain_orthogonalize(g, steps):
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(steps):
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return (x.transpose(1, 2) if tall else x).to(g.dtype)


# ---------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "quantize":
        x, fmt, pow2 = state["x"], case["format"], case["pow2"]
        if case["block"] == "pair":
            return _plain_quantize(x, "row", fmt, pow2) + _plain_quantize(x, "column", fmt, pow2)
        return _plain_quantize(x, case["block"], fmt, pow2)
    if case["op"] == "product":
        return _plain_product(case, state["operands"], state.get("d"))
    return _plain_orthogonalize(state["g"], case["steps"])


def _run_own(case, state):
    import dense_fp32_matrix_08_gb300 as sg
    if case["op"] == "quantize":
        kw = dict(dtype=FORMAT[case["format"]], pow2=case["pow2"])
        if case["block"] == "pair":
            return sg.f8_quantize_pair(state["x"], **kw)
        block = {"row": (1, 128), "column": (128, 1), "square": (128, 128)}[case["block"]]
        return sg.f8_quantize(state["x"], block, **kw)
    if case["op"] == "product":
        qa, sa, _, ta, qb, sb, _, tb = state["operands"]
        if "d" in state:
            return sg.f8_matmul(qa, sa, qb, sb, transa=ta, transb=tb, beta=1.0, out=state["d"])
        return sg.f8_matmul(qa, sa, qb, sb, transa=ta, transb=tb,
                            out_dtype=TYPE[case["type"]])
    return sg.orthogonalize(state["g"], steps=case["steps"], coefficients=COEFFICIENTS, eps=EPS)


# ---------------------------------------------------------------------------- least work

def work(case):
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        row = r * c + 4 * r * -(-c // BLOCK)
        column = r * c + 4 * c * -(-r // BLOCK)
        out = {"row": row, "column": column, "pair": row + column,
               "square": r * c + 4 * -(-r // BLOCK) * -(-c // BLOCK)}[case["block"]]
        passes = 2 if case["block"] == "pair" else 1
        return {"bytes": r * c * SIZE[case["type"]] + out, "flops": 2 * r * c * passes}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        sb = kb * n if case["kind"] == "wgrad" else kb * -(-n // BLOCK)
        d = m * n * SIZE[case["type"]] * (2 if case["kind"] == "wgrad" else 1)
        return {"bytes": m * k + k * n + 4 * (m * kb + sb) + d, "flops": 2 * m * n * k}
    s, l = sorted((case["m"], case["n"]))
    each = s * s * l + s * s * s + 2 * s * s * l  # S and S^2 are symmetric: half of each
    return {"bytes": 2 * case["batch"] * s * l * SIZE[case["type"]],
            "flops": case["batch"] * case["steps"] * each}


# ---------------------------------------------------------------------------- 64 bits

def _exact_round(v, fmt):
    """v rounded to the nearest number of the format, ties to even, limited to its range."""
    bits, least = (3, -6) if fmt == "e4m3" else (2, -14)
    _, power = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp_min(power - 1, least) - bits)
    return (torch.round(v / step) * step).clamp(-LARGEST[fmt], LARGEST[fmt])


def _exact_quantize(x, br, bc, fmt, pow2):
    rows, cols = x.shape
    nr, nc = (rows + br - 1) // br, (cols + bc - 1) // bc
    x = torch.nn.functional.pad(x.double(), (0, nc * bc - cols, 0, nr * br - rows))
    x = x.reshape(nr, br, nc, bc)
    s = torch.maximum(x.abs().amax(3, True).amax(1, True) / LARGEST[fmt],
                      torch.tensor(2.0 ** -126, dtype=torch.float64, device=x.device))
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    q = _exact_round(x / s, fmt).reshape(nr * br, nc * bc)[:rows, :cols]
    return q, s.reshape(nr, nc)


def _exact_values(q, s, block):
    r = torch.arange(q.shape[0], device=q.device)
    c = torch.arange(q.shape[1], device=q.device)
    r = r if block == "row" else r // BLOCK
    c = c if block == "column" else c // BLOCK
    return q.double() * s.double()[r[:, None], c[None, :]]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        sides = {"row": [(1, 128)], "column": [(128, 1)], "square": [(128, 128)],
                 "pair": [(1, 128), (128, 1)]}[case["block"]]
        out = []
        for br, bc in sides:
            out += _exact_quantize(state["x"], br, bc, case["format"], case["pow2"])
        return tuple(out)
    if case["op"] == "product":
        qa, sa, ba, ta, qb, sb, bb, tb = state["operands"]
        a, b = _exact_values(qa, sa, ba), _exact_values(qb, sb, bb)
        y = torch.matmul(a.mT if ta else a, b.mT if tb else b)
        return y + state["d"].double() if "d" in state else y
    g = state["g"].double()
    a, b, c = COEFFICIENTS
    x = g / (torch.linalg.matrix_norm(g, keepdim=True) + EPS)
    for _ in range(case["steps"]):
        if g.shape[1] <= g.shape[2]:
            s = torch.bmm(x, x.mT)
            x = a * x + b * torch.bmm(s, x) + c * torch.bmm(s, torch.bmm(s, x))
        else:
            s = torch.bmm(x.mT, x)
            x = a * x + b * torch.bmm(x, s) + c * torch.bmm(torch.bmm(x, s), s)
    return x
