"""A small training loop over the low-precision operators, as they are used
together: linear layers whose products run on block-scaled 8-bit operands,
fp32 master weights and gradients, and a momentum that is orthogonalised before
it is applied.

    python -m dense_fp32_matrix_row_amd.lowp_training --steps 60

fits a two-layer network to a fixed random one and prints the loss as it falls,
then runs the trained network on single tokens.
"""

from __future__ import annotations

import argparse
import math

from . import blockfp8, orthogonal


class Layer:
    """An out x in weight: the fp32 master, its momentum, and the 8-bit forms for
    the forward and the backward product, remade after every update."""

    def __init__(self, weight, scale):
        import torch
        self.master = weight
        self.momentum = torch.zeros_like(weight)
        self.gradient = torch.zeros_like(weight)
        self.scale = scale
        self.quantize()

    def quantize(self):
        self.w, self.wt = blockfp8.quantize_both(self.master, blockfp8.BLOCK, self.scale)

    def update(self, rate, decay=0.9):
        """Moves the weight against its orthogonalised momentum, whose singular
        values are all about 1: by `rate` in spectral norm, whatever the
        gradient's size."""
        self.momentum.mul_(decay).add_(self.gradient)
        self.master.sub_(orthogonal.orthogonalize(self.momentum), alpha=rate)
        self.gradient.zero_()
        self.quantize()


class Network:
    """y = W2 relu(W1 x) for rows of tokens."""

    def __init__(self, inputs, hidden, outputs, seed=0, scale=None, device="cuda"):
        import torch
        g = torch.Generator(device=device).manual_seed(seed)
        make = lambda o, i: torch.randn(o, i, generator=g, device=device) / math.sqrt(i)  # noqa: E731
        scale = scale or torch.float32
        self.layers = Layer(make(hidden, inputs), scale), Layer(make(outputs, hidden), scale)

    def forward(self, x):
        """The outputs, and what backward needs."""
        one, two = self.layers
        h, xt = blockfp8.linear_forward(x, one.w)
        y, ht = blockfp8.linear_forward(h.relu_(), two.w)
        return y, (xt, h, ht)

    def backward(self, dy, saved):
        """Adds the weights' gradients to Layer.gradient."""
        xt, h, ht = saved
        one, two = self.layers
        dh, _ = blockfp8.linear_backward(dy, ht, two.wt, dw=two.gradient)
        blockfp8.linear_backward(dh * (h > 0), xt, one.wt, dw=one.gradient)

    def infer(self, x):
        """The outputs alone, for any number of tokens."""
        one, two = self.layers
        h = blockfp8.gemm(blockfp8.quantize(x, 1, one.scale), one.w, out_dtype=x.dtype)
        return blockfp8.gemm(blockfp8.quantize(h.relu_(), 1, two.scale), two.w, out_dtype=x.dtype)


def train(steps=60, tokens=512, inputs=256, hidden=384, outputs=130, rate=0.05, seed=0, scale=None):
    """Trains a Network on a fixed random one's outputs; returns it and the losses."""
    import torch
    network = Network(inputs, hidden, outputs, seed, scale)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    target = randn(outputs, inputs) / math.sqrt(inputs)
    losses = []
    for step in range(steps):
        x = randn(tokens, inputs)
        want = x @ target.T
        y, saved = network.forward(x.bfloat16())
        error = y.float() - want
        losses.append(error.square().mean())
        network.backward((error * (2 / error.numel())).bfloat16(), saved)
        for layer in network.layers:
            layer.update(rate * (1 - step / steps))
    return network, [float(loss) for loss in losses]


def main(argv=None):
    import torch
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--scale", choices=("f32", "e8m0"), default="f32", help="the type of the blocks' scales")
    args = parser.parse_args(argv)
    network, losses = train(args.steps, scale=torch.float32 if args.scale == "f32" else torch.float8_e8m0fnu)
    for step in range(0, len(losses), max(len(losses) // 10, 1)):
        print(f"step {step:4d}  loss {losses[step]:.5f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.5f}")
    x = torch.randn(8, 256, device="cuda").bfloat16()
    together = network.infer(x)
    apart = torch.cat([network.infer(x[i:i + 1]) for i in range(8)])
    print(f"eight tokens at once and one by one differ by {float((together.float() - apart.float()).abs().max()):.2e}")


if __name__ == "__main__":
    main()
