"""Two linear layers trained in 8-bit floating point with orthogonalised updates.

Activations, weights and gradients are quantised to E4M3 with one float32 scale
per 128 values (weights: per 128 x 128), every product runs on those codes, the
weights' gradients are summed into float32, and the update is the momentum's
Newton-Schulz orthogonalisation.  Synthetic data; prints the loss.

    python examples/train_block8.py [--steps 60] [--width 512] [--tokens 2048]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from stride_layouts_lds_amd import api  # noqa: E402


def product(a, b, dtype=torch.bfloat16):
    """a b^T of two (codes, scales) pairs."""
    return api.gemm(a[0], b[0], sfa=a[1], sfb=b[1], block_k=128, dtype=dtype)


class Linear:
    """y = x W^T with W (out, in) kept in float32."""

    def __init__(self, n_in, n_out, gen):
        self.w = torch.randn(n_out, n_in, generator=gen, device="cuda") * n_in ** -0.5
        self.momentum = torch.zeros_like(self.w)

    def forward(self, x):
        # one read of x and of W serves the forward product and both gradients
        q, s, self.xt, self.xts = api.quantize(x, transposed=True)
        wq, ws, self.wt, self.wts = api.quantize(self.w, block_rows=128, transposed=True)
        return product((q, s), (wq, ws))

    def backward(self, g):
        """W's gradient (float32) and x's."""
        q, s, qt, st = api.quantize(g, transposed=True)
        return product((qt, st), (self.xt, self.xts), torch.float32), product((q, s), (self.wt, self.wts))

    def step(self, grad, lr):
        self.momentum.mul_(0.9).add_(grad)
        update = api.orthogonalize(self.momentum)
        m, n = self.w.shape
        self.w.add_(update, alpha=-lr * max(1.0, m / n) ** 0.5)


def train(steps=60, width=512, tokens=2048, lr=0.02, seed=0, report=None):
    """The losses of the steps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher = [Linear(width, 2 * width, gen), Linear(2 * width, width, gen)]
    layers = [Linear(width, 2 * width, gen), Linear(2 * width, width, gen)]
    losses = []
    for i in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
        want = torch.relu(x.float() @ teacher[0].w.t()) @ teacher[1].w.t()
        h = layers[0].forward(x)
        y = layers[1].forward(torch.relu(h))
        e = y.float() - want
        losses.append(float(e.square().mean()))
        gw1, gh = layers[1].backward((e * (2.0 / tokens)).bfloat16())
        gw0, _ = layers[0].backward(gh * (h > 0))
        layers[1].step(gw1, lr)
        layers[0].step(gw0, lr)
        if report and (i % report == 0 or i + 1 == steps):
            print(f"step {i:4d}  loss {losses[-1]:.5f}", flush=True)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--lr", type=float, default=0.02)
    args = ap.parse_args()
    train(args.steps, args.width, args.tokens, args.lr, report=10)
