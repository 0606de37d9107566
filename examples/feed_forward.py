"""A pre-norm feed-forward block on the library's dense operators: a training
step (forward, gradients, update), single tokens, and a prompt with int8 weights.

    y = x + w2 act(w1 norm(x) + b1) + b2

    python examples/feed_forward.py --rows 8192 --width 2048 --hidden 8192
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_convolution_forward_amd as ci8  # noqa: E402


class FeedForward:
    """Parameters, and the calls that use them.  What `forward` keeps for
    `backward` is returned and not stored."""

    def __init__(self, width, hidden, dtype=torch.bfloat16, activation="gelu_tanh", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s, scale: (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)  # noqa: E731
        self.activation = activation
        self.params = {
            "gamma": torch.ones(width, dtype=dtype, device="cuda"),
            "beta": torch.zeros(width, dtype=dtype, device="cuda"),
            "w1": normal(hidden, width, scale=width ** -0.5),
            "b1": normal(hidden, scale=0.02),
            "w2": normal(width, hidden, scale=hidden ** -0.5),
            "b2": normal(width, scale=0.02),
        }
        self.quantised = None

    def __call__(self, x):
        """One pass without gradients: three launches."""
        p = self.params
        h, _, _ = ci8.layer_norm(x, p["gamma"], p["beta"])
        a = ci8.linear(h, p["w1"], p["b1"], activation=self.activation)
        return ci8.linear(a, p["w2"], p["b2"], residual=x)

    def forward(self, x):
        """(y, what backward takes)."""
        p = self.params
        h, mean, rstd = ci8.layer_norm(x, p["gamma"], p["beta"])
        z = torch.empty(*x.shape[:-1], p["w1"].shape[0], dtype=x.dtype, device=x.device)
        a = ci8.linear(h, p["w1"], p["b1"], activation=self.activation, preact=z)
        return ci8.linear(a, p["w2"], p["b2"], residual=x), (x, mean, rstd, h, z, a)

    def backward(self, dy, kept):
        """(dx, gradients by name)."""
        x, mean, rstd, h, z, a = kept
        p, g = self.params, {}
        da, g["w2"], g["b2"] = ci8.linear_backward(dy, a, p["w2"])
        dh, g["w1"], g["b1"] = ci8.linear_backward(da, h, p["w1"], preact=z, activation=self.activation)
        dx, g["gamma"], g["beta"] = ci8.layer_norm_backward(dh, x, p["gamma"], mean, rstd)
        return dx + dy, g  # dy also goes past the block, along the residual

    def step(self, grads, rate):
        for name, p in self.params.items():
            p.sub_(grads[name], alpha=rate)
        self.quantised = None

    def quantise(self):
        """w1 as int8 rows with a scale each, laid out once."""
        w = self.params["w1"].float()
        scale = w.abs().amax(1).clamp_min(torch.finfo(torch.float32).tiny) / 127
        self.quantised = ((w / scale[:, None]).round().to(torch.int8), scale)

    def prompt_i8(self, x):
        """The pass with the widening product in int8: layer norm writes the
        rows and scales that the product takes."""
        if self.quantised is None:
            self.quantise()
        p = self.params
        w, w_scale = self.quantised
        q, x_scale = ci8.layer_norm_i8(x, p["gamma"], p["beta"])
        a = ci8.linear(q, w, p["b1"], activation=self.activation, x_scale=x_scale, w_scale=w_scale, out_dtype=x.dtype)
        return ci8.linear(a, p["w2"], p["b2"], residual=x)


def milliseconds(f, n=10):
    f()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(n):
        f()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / n


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=None, help="of the updates (default: 4 / hidden)")
    args = ap.parse_args(argv)
    # the loss's largest curvature is about hidden / 6: the activations' means add up over the hidden dimension
    rate = 4 / args.hidden if args.rate is None else args.rate

    # fit the block to another one's outputs
    block, teacher = FeedForward(args.width, args.hidden), FeedForward(args.width, args.hidden, seed=1)
    x = torch.randn(args.rows, args.width, device="cuda").to(torch.bfloat16)
    target = teacher(x)

    def loss_and_gradient(y):
        d = y.float() - target.float()
        return d.square().mean(), (d * (2 / args.rows)).to(y.dtype)  # of the sum over columns

    def train_step():
        y, kept = block.forward(x)
        loss, dy = loss_and_gradient(y)
        _, grads = block.backward(dy, kept)
        block.step(grads, rate)
        return loss

    losses = [float(train_step()) for _ in range(args.steps)]
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f} in {args.steps} steps")
    y = block(x)
    y8 = block.prompt_i8(x)
    off = float((y8.float() - y.float()).norm() / (y.float() - x.float()).norm())
    print(f"int8 widening product: the block's output is off by {off:.4f} of its norm")
    print(f"training step {milliseconds(train_step):.3f} ms, prompt {milliseconds(lambda: block(x)):.3f} ms, "
          f"int8 prompt {milliseconds(lambda: block.prompt_i8(x)):.3f} ms, one token "
          f"{milliseconds(lambda: block(x[:1])):.4f} ms")
    return losses, off


if __name__ == "__main__":
    main()
