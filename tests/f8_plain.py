"""Plain 64-bit forms of the 8-bit block-scaled operators, for the tests: block scales, rounding
to the two formats, and the product, from their definitions, on CPU tensors."""
import torch

LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
FORMAT = {torch.float8_e4m3fn: (3, -6), torch.float8_e5m2: (2, -14)}  # fraction bits, least exponent


def f32(x):
    """Round 64-bit values to FP32 (a quotient of two FP32 numbers rounded to 53 bits first rounds
    to the same FP32 number as the quotient itself: 53 >= 2 * 24 + 2)."""
    return x.to(torch.float32).double()


def round_to(v, dtype):
    bits, least = FORMAT[dtype]
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(least) - bits)
    return (torch.round(v / step) * step).clamp(-LARGEST[dtype], LARGEST[dtype])


def block_index(n, size):
    return torch.arange(n) // size


def quantize(x, block, dtype, pow2):
    """(values of q, scales), both 64-bit."""
    x = x.double()
    rows, cols = x.shape
    br, bc = block
    nr, nc = -(-rows // br), -(-cols // bc)
    y = torch.zeros(nr * br, nc * bc, dtype=torch.float64)
    y[:rows, :cols] = x.abs()
    top = y.view(nr, br, nc, bc).amax(dim=(1, 3))
    s = f32(top / LARGEST[dtype]).clamp_min(2.0 ** -126)
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    q = round_to(f32(x / s[block_index(rows, br)][:, block_index(cols, bc)]), dtype)
    return q, s


def values(q, scale):
    """The numbers a quantised matrix stands for (64-bit)."""
    rows, cols = q.shape
    br = 1 if scale.shape[0] == rows else 128
    bc = 1 if scale.shape[1] == cols else 128
    return q.double() * scale.double()[block_index(rows, br)][:, block_index(cols, bc)]
