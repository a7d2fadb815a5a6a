"""A residual block y = x + W2 relu(W1 norm(x)), trained with the 8-bit products and served in 8-bit
integers.

    python examples/normed_mlp.py [--tokens 2048] [--width 512] [--steps 30]

One step of training runs
    h = norm(x)                     with the statistics that its gradients take        (layer_norm)
    the products of both layers and their gradients, added up over batches              (Linear8)
    dx, and the gradients of the norm's weight and bias, added up in FP32    (layer_norm_backward)
    all gradients times min(1, limit / their norm)                               (clip_grad_norm)
    the orthogonalised update of both weights                                       (orthogonalize)
Serving quantises the weights once, a scale for each output, and then, for one token or many, runs
    h = norm(x); a = relu(h W1^T); y = x + a W2^T        (layer_norm, i8_quantize, i8_linear)
with the residual added in the product's own last step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from f8_linear_layer import Linear8, problem, sg  # noqa: E402


class Block:
    def __init__(self, w1, w2):
        self.first, self.second = Linear8(w1), Linear8(w2)
        width = w1.shape[1]
        self.weight, self.bias = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
        self.dweight, self.dbias = torch.zeros_like(self.weight), torch.zeros_like(self.bias)
        self.batches = 0  # added to dweight and dbias since the last update

    def forward(self, x):
        self.x = x
        h, self.mean, self.rstd = sg.layer_norm(x, self.weight, self.bias, stats=True)
        self.a = self.first.forward(h).relu_()
        return x + self.second.forward(self.a)

    def backward(self, dy):
        """Adds one batch's gradients; returns that of x."""
        da = self.second.backward(dy)
        self.dh = self.first.backward(da * (self.a > 0))
        dx, _, _ = sg.layer_norm_backward(self.dh, self.x, self.mean, self.rstd, self.weight, dweight=self.dweight,
                                          dbias=self.dbias, beta=1.0 if self.batches else 0.0)
        self.batches += 1
        return dx.add_(dy)

    def update(self, rate, limit):
        """Clips the gradients, applies them and returns their norm before that (on the device)."""
        norm = sg.clip_grad_norm([self.first.grad, self.second.grad, self.dweight, self.dbias], limit)
        self.first.update(rate)
        self.second.update(rate)
        self.weight.sub_(self.dweight, alpha=rate)
        self.bias.sub_(self.dbias, alpha=rate)
        self.batches = 0
        return norm

    def quantize(self):
        """What serving keeps: the norm's parameters and both weights in 8-bit integers."""
        return Served(self.weight, self.bias, sg.i8_quantize(self.first.weight), sg.i8_quantize(self.second.weight))


class Served:
    def __init__(self, weight, bias, first, second):
        self.weight, self.bias, self.first, self.second = weight.clone(), bias.clone(), first, second

    def __call__(self, x):
        h = sg.layer_norm(x, self.weight, self.bias)
        a = sg.i8_linear(*sg.i8_quantize(h), *self.first, out_dtype=x.dtype).relu_()
        return sg.i8_linear(*sg.i8_quantize(a), *self.second, beta=1.0, out=x.clone())


def train(block, x, target, steps, rate, limit, batches=2):
    """Losses and gradient norms before each update."""
    losses, norms = [], []
    for step in range(steps):
        loss = 0.0
        for a, b in zip(x.chunk(batches), target.chunk(batches)):
            e = block.forward(a).float() - b.float()
            loss = loss + 0.5 * e.square().mean() / batches
            block.backward((e / e.numel()).to(x.dtype))
        losses.append(loss)
        norms.append(block.update(rate * (1.0 - step / steps), limit))
    return [v.item() for v in losses], [v.item() for v in norms]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--rate", type=float, default=0.05)
    ap.add_argument("--limit", type=float, default=1.0)
    args = ap.parse_args()
    x, target, w1, w2 = problem(args.tokens, args.width)
    block = Block(w1, w2)
    losses, norms = train(block, x, target, args.steps, args.rate, args.limit)
    every = max(1, args.steps // 10)
    print("loss", " ".join(f"{v:.4f}" for v in losses[::every]))
    print("norm", " ".join(f"{v:.2e}" for v in norms[::every]))
    serve, trained = block.quantize(), block.forward(x)
    one, all_ = serve(x[:1]), serve(x)
    print(f"one token against the batch: {(one - all_[:1]).abs().max().item():.3g} apart; served against trained: "
          f"{(all_.float() - trained.float()).norm().item() / trained.float().norm().item():.3g} of the norm")


if __name__ == "__main__":
    main()
