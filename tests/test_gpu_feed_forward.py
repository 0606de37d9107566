"""The feed-forward example: its gradients against the same block in 64 bits,
its training, and its int8 form."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(p, x):
    """The block from its definition, in the type of x."""
    c = x - x.mean(-1, keepdim=True)
    h = c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
    z = h @ p["w1"].t() + p["b1"]
    a = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return x + a @ p["w2"].t() + p["b2"]


@pytest.mark.parametrize("rows,width,hidden", [((1,), 64, 256), ((37,), 136, 520), ((3, 50), 101, 77), ((600,), 256, 1024)])
def test_block_and_gradients(ff, rows, width, hidden):
    """Along the block a handful of values are rounded to 16 bits (h, z, a, da,
    g, dh and the outputs), each by at most 2^-8 of itself; errors of different
    values are independent, so in the norm an output is off by a few 2^-8: 2^-5
    leaves four times that."""
    block = ff.FeedForward(width, hidden, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(*rows, width, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(*rows, width, generator=g, device="cuda").to(torch.bfloat16)
    y, kept = block.forward(x)
    dx, grads = block.backward(dy, kept)
    assert torch.equal(y, block(x))

    p = {k: v.double().cpu().requires_grad_() for k, v in block.params.items()}
    xd = x.double().cpu().requires_grad_()
    want = plain(p, xd)
    want.backward(dy.double().cpu())
    for name, got, ref in [("y", y, want.detach()), ("dx", dx, xd.grad)] + [(k, grads[k], p[k].grad) for k in p]:
        off = float((got.double().cpu() - ref).norm() / ref.norm())
        assert off < 2 ** -5, (name, off)


def test_training_and_int8(ff):
    """The loss falls; the int8 product (rows and weights off by at most half a
    step of 1/127 of their largest value, about four standard deviations: 1 %
    of a standard deviation each) leaves the block's output within 5 %."""
    losses, off = ff.main(["--rows", "512", "--width", "256", "--hidden", "1024", "--steps", "10"])
    assert losses[-1] < losses[0] and all(math.isfinite(v) for v in losses)
    assert off < 0.05
