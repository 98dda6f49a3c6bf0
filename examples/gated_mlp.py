"""A gated MLP trained in bf16 and served in 8 bits, with the library's own operators.

y = (silu(x Wg) * (x Wu)) Wd is fitted to a fixed random teacher of the same shape by gradient descent
with float32 master weights: swiglu_forward and matmul forward, matmul_backward and swiglu_backward
back. The trained weights are then quantised once, row by row in the nn.Linear layout, and
tokens are served with i8_swiglu_linear and i8_linear, in batches and one at a time.

    python examples/gated_mlp.py [--tokens 512] [--width 512] [--hidden 1376] [--steps 60]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemv_layers_amd as g  # noqa: E402


class GatedMLP:
    """Gate/up weight B (width x 2 hidden, gate columns first) and down weight D (hidden x width)."""

    def __init__(self, width, hidden, gen):
        self.B = torch.randn(width, 2 * hidden, generator=gen, device="cuda") * width**-0.5
        self.D = torch.randn(hidden, width, generator=gen, device="cuda") * hidden**-0.5

    def bf16(self):
        return self.B.bfloat16(), self.D.bfloat16()

    def forward(self, x):
        b, d = self.bf16()
        h, gu = g.swiglu_forward(x, b)
        return g.matmul(h, d), (x, b, d, h, gu)

    def backward(self, dy, saved):
        """(dB, dD) for the loss gradient dy; the input's gradient is not needed here."""
        x, b, d, h, gu = saved
        dh, dD = g.matmul_backward(dy, h, d)
        _, dB, _ = g.swiglu_backward(dh, gu, x, b, need_dA=False, inplace=True)
        return dB, dD


class ServedMLP:
    """The 8-bit form: codes and scales of the transposed weights, made once."""

    def __init__(self, mlp):
        b, d = mlp.bf16()
        self.gate_up = g.i8_quantize(b.t().contiguous())
        self.down = g.i8_quantize(d.t().contiguous())

    def __call__(self, x):
        return g.i8_linear(g.i8_swiglu_linear(x, *self.gate_up), *self.down)


def train(tokens, width, hidden, steps, lr=0.1, seed=0):
    """Returns (model, losses)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher, model = GatedMLP(width, hidden, gen), GatedMLP(width, hidden, gen)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
        target, _ = teacher.forward(x)
        y, saved = model.forward(x)
        diff = y.float() - target.float()
        losses.append(diff.square().mean())
        dB, dD = model.backward((diff * (2 / tokens)).bfloat16(), saved)
        model.B -= lr * dB.float()
        model.D -= lr * dD.float()
    return model, [float(v) for v in losses]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1376)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args(argv)
    g.gemm_init(torch.cuda.current_device())
    model, losses = train(a.tokens, a.width, a.hidden, a.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    want, _ = model.forward(x)
    served = ServedMLP(model)
    got = served(x)
    one = torch.cat([served(x[i:i + 1]) for i in range(4)])
    error = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"8-bit serving: relative error {error:.4f}; one token at a time gives the same bits: "
          f"{bool(torch.equal(one, got[:4]))}")
    return losses, error, torch.equal(one, got[:4])


if __name__ == "__main__":
    main()
