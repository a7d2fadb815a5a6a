"""Two linear layers trained and served with the 8-bit operators and the orthogonalised update.

    python examples/f8_linear_layer.py [--tokens 2048] [--width 512] [--steps 30]

Each layer keeps its weight in FP32 and an 8-bit copy of it that is renewed after every update.
One step of training runs, for each layer:
    y  = x W^T      x by rows of 128, W by 128 x 128 blocks                  (f8_matmul, NT)
    dx = dy W       dy by rows of 128, the same copy of W                    (f8_matmul, NN)
    dW += dy^T x    both by columns of 128 tokens, added up in FP32          (f8_matmul, TN)
    W  = (1 - rate decay) W - rate scale orthogonalised(momentum)            (orthogonalize)
x and dy are read once each for both of their forms (f8_quantize_pair). Serving is the first product
alone, for as few as one token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_matrix_08_gb300 as sg  # noqa: E402


class Linear8:
    """y = x W^T with W of (outputs, inputs)."""

    def __init__(self, weight):
        self.weight = weight.float().contiguous()
        self.grad = torch.empty_like(self.weight)
        self.momentum = torch.zeros_like(self.weight)
        self.batches = 0  # added to grad since the last update
        self.renew()

    def renew(self):
        self.w8, self.w8_scale = sg.f8_quantize(self.weight, (128, 128))

    def serve(self, x):
        q, scale = sg.f8_quantize(x)
        return sg.f8_matmul(q, scale, self.w8, self.w8_scale, transb=True)

    def forward(self, x):
        q, scale, *self.x_columns = sg.f8_quantize_pair(x)
        return sg.f8_matmul(q, scale, self.w8, self.w8_scale, transb=True)

    def backward(self, dy, need_dx=True):
        q, scale, *dy_columns = sg.f8_quantize_pair(dy)
        sg.f8_matmul(*dy_columns, *self.x_columns, transa=True, out=self.grad,
                     beta=1.0 if self.batches else 0.0)
        self.batches += 1
        return sg.f8_matmul(q, scale, self.w8, self.w8_scale) if need_dx else None

    def update(self, rate, momentum=0.9, decay=0.0):
        self.momentum.mul_(momentum).add_(self.grad)
        rows, cols = self.weight.shape
        sg.orthogonalize(self.momentum, alpha=-rate * max(1.0, rows / cols) ** 0.5,
                         beta=1.0 - rate * decay, out=self.weight)
        self.batches = 0
        self.renew()


class Pair:
    """y = relu(x W1^T) W2^T, fitted to targets by least squares."""

    def __init__(self, w1, w2):
        self.first, self.second = Linear8(w1), Linear8(w2)

    def serve(self, x):
        return self.second.serve(self.first.serve(x).relu_())

    def accumulate(self, x, target):
        """Adds one batch's gradient; returns its loss (on the device)."""
        h = self.first.forward(x).relu_()
        e = self.second.forward(h).float() - target.float()
        dh = self.second.backward((e / e.numel()).to(x.dtype))
        self.first.backward(dh * (h > 0), need_dx=False)
        return 0.5 * e.square().mean()

    def update(self, rate):
        self.first.update(rate)
        self.second.update(rate)


def problem(tokens, width, seed=0, dtype=torch.bfloat16):
    """Inputs, targets of a known pair of layers, and the weights to start from."""
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, scale=1.0):
        return scale * torch.randn(*shape, generator=g)

    x = rand(tokens, width)
    t1, t2 = rand(2 * width, width, scale=width ** -0.5), rand(width, 2 * width, scale=width ** -0.5)
    target = (x @ t1.t()).relu() @ t2.t()
    w1, w2 = rand(2 * width, width, scale=width ** -0.5), rand(width, 2 * width, scale=width ** -0.5)
    return x.to(dtype).cuda(), target.to(dtype).cuda(), w1.cuda(), w2.cuda()


def train(model, x, target, steps, rate, batches=2):
    """Losses before each update; a step adds up the gradients of `batches` parts of the tokens."""
    losses = []
    for step in range(steps):
        parts = zip(x.chunk(batches), target.chunk(batches))
        losses.append(sum(model.accumulate(a, b) for a, b in parts) / batches)
        model.update(rate * (1.0 - step / steps))
    return [loss.item() for loss in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--rate", type=float, default=0.05)
    args = ap.parse_args()
    x, target, w1, w2 = problem(args.tokens, args.width)
    model = Pair(w1, w2)
    losses = train(model, x, target, args.steps, args.rate)
    print("loss", " ".join(f"{v:.4f}" for v in losses[::max(1, args.steps // 10)]))
    one, all_ = model.serve(x[:1]), model.serve(x)
    print(f"one token against the batch: {(one - all_[:1]).abs().max().item():.3g} apart, "
          f"largest output {all_[:1].abs().max().item():.3g}")


if __name__ == "__main__":
    main()
