"""A stack of feed-forward blocks with their products in 8-bit floating point: a
training step (forward, gradients, clipping, update) and single tokens.

    r = x + gate norm(h) post,  y = norm(r) gamma + beta     between the blocks, in one pass
    h = w2 act(w1 y + b1) + b2                               operands in 8 bits, a scale for each block of 128

    python examples/feed_forward_fp8.py --rows 8192 --width 2048 --hidden 8192
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_convolution_forward_amd as ci8  # noqa: E402


class Block:
    """The norm before a block, fused with the residual connection after the one before it (`h` of which
    is None for the first), and the block.  What `forward` keeps for `backward` is returned and not stored."""

    def __init__(self, width, hidden, first, dtype=torch.bfloat16, activation="gelu_tanh", norm="rms", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s, scale: (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)  # noqa: E731
        self.activation, self.norm = activation, norm
        self.params = {
            "gamma": torch.ones(width, dtype=dtype, device="cuda"),
            "beta": torch.zeros(width, dtype=dtype, device="cuda"),
            "w1": normal(hidden, width, scale=width ** -0.5),
            "b1": normal(hidden, scale=0.02),
            "w2": normal(width, hidden, scale=hidden ** -0.5),
            "b2": normal(width, scale=0.02),
        }
        if not first:
            self.params["gate"] = normal(width, scale=0.5)
            self.params["post"] = torch.ones(width, dtype=dtype, device="cuda")
        self.quantise()

    def quantise(self):
        """The weights in 8 bits and their transposes, laid out once for all calls until the next update."""
        for name in ("w1", "w2"):
            setattr(self, name, ci8.quantize_fp8(self.params[name], block="tiles", transposed=True))

    def between(self):
        p = self.params
        return dict(weight=p["gamma"], gate=p.get("gate"), post_weight=p.get("post"), norm=self.norm)

    def __call__(self, x, h):
        """(r, h) without gradients: five launches."""
        p = self.params
        r, q, s = ci8.residual_norm_fp8(x, h, bias=p["beta"], **self.between())
        a = ci8.linear_fp8(q, self.w1[0], s, self.w1[1], p["b1"], activation=self.activation)
        q, s = ci8.quantize_fp8(a)
        return r, ci8.linear_fp8(q, self.w2[0], s, self.w2[1], p["b2"])

    def forward(self, x, h):
        """(r, h, what backward takes)."""
        p = self.params
        r, y, stats = ci8.residual_norm(x, h, bias=p["beta"], **self.between())
        yq, ys, yt, yts = ci8.quantize_fp8(y, transposed=True)
        z = torch.empty(*x.shape[:-1], p["w1"].shape[0], dtype=x.dtype, device=x.device)
        a = ci8.linear_fp8(yq, self.w1[0], ys, self.w1[1], p["b1"], activation=self.activation, preact=z)
        aq, as_, at, ats = ci8.quantize_fp8(a, transposed=True)
        return r, ci8.linear_fp8(aq, self.w2[0], as_, self.w2[1], p["b2"]), (r, h, stats, yt, yts, z, at, ats)

    def backward(self, dr, dh, kept):
        """(gradient of x, of h, gradients by name) from those of r (None: zero) and of the block's output."""
        r, h, stats, yt, yts, z, at, ats = kept
        g = {}
        da, g["w2"], g["b2"] = ci8.linear_fp8_backward(dh, at, ats, self.w2[2], self.w2[3])
        dy, g["w1"], g["b1"] = ci8.linear_fp8_backward(da, yt, yts, self.w1[2], self.w1[3], preact=z,
                                                       activation=self.activation)
        dx, dh, g["gamma"], g["beta"], gate, post = ci8.residual_norm_backward(dr, dy, r, h, stats, **self.between())
        if h is not None:
            g["gate"], g["post"] = gate, post
        return dx, dh, g


class Stack:
    def __init__(self, blocks, width, hidden, seed=0, **kw):
        self.blocks = [Block(width, hidden, i == 0, seed=seed + i, **kw) for i in range(blocks)]

    def __call__(self, x):
        h = None
        for b in self.blocks:
            x, h = b(x, h)
        return x + h

    def forward(self, x):
        kept, h = [], None
        for b in self.blocks:
            x, h, k = b.forward(x, h)
            kept.append(k)
        return x + h, kept

    def backward(self, dy, kept):
        """(dx, gradients of each block)."""
        dr, dh, grads = dy, dy, []
        for b, k in zip(reversed(self.blocks), reversed(kept)):
            dr, dh, g = b.backward(dr, dh, k)
            grads.insert(0, g)
        return dr, grads

    def step(self, grads, rate, max_norm):
        """Clips the gradients of all blocks together and updates; returns their norm."""
        pairs = [(p, g[name]) for b, g in zip(self.blocks, grads) for name, p in b.params.items()]
        norm = ci8.clip_grad_norm([g for _, g in pairs], max_norm)
        for p, g in pairs:
            p.sub_(g, alpha=rate)
        for b in self.blocks:
            b.quantise()
        return norm


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
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--rate", type=float, default=1e-3)
    ap.add_argument("--max-norm", type=float, default=1.0)
    args = ap.parse_args(argv)
    stack, teacher = (Stack(args.blocks, args.width, args.hidden, seed=s) for s in (0, 100))
    x = torch.randn(args.rows, args.width, device="cuda").to(torch.bfloat16)
    target = teacher(x)

    def train_step():
        y, kept = stack.forward(x)
        d = y.float() - target.float()
        _, grads = stack.backward((d * (2 / args.rows)).to(y.dtype), kept)
        return d.square().mean(), stack.step(grads, args.rate, args.max_norm)

    losses, norms = zip(*((float(a), float(b)) for a, b in (train_step() for _ in range(args.steps))))
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}, gradient norm {norms[0]:.3f} -> {norms[-1]:.3f} in {args.steps} steps")
    print(f"training step {milliseconds(train_step):.3f} ms, prompt {milliseconds(lambda: stack(x)):.3f} ms, "
          f"one token {milliseconds(lambda: stack(x[:1])):.4f} ms")
    return losses, norms


if __name__ == "__main__":
    main()
