"""The entries around a block in 8-bit floating point beside automatic
differentiation, on other streams, recorded into graphs, and run together as a
training step and on single tokens."""
import importlib.util
import os
from types import SimpleNamespace

import pytest
import torch

from tests import block_reference as ref
from tests.dense_reference import act, slope

pytestmark = pytest.mark.gpu

BF16, E4 = torch.bfloat16, torch.float8_e4m3fn
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("feed_forward_fp8", os.path.join(ROOT, "examples", "feed_forward_fp8.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def operands(ci8, m, seed=61, d=256, n=384):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    t = dict(x=r(m, d), h=r(m, d), gamma=r(d), beta=r(d), gate=r(d), post=r(d), bias=r(n), res=r(m, n), dy=r(m, n), z=r(m, n),
             dr=r(m, d), out=r(m, n))
    t["q"], t["s"], t["qt"], t["st"] = ci8.quantize_fp8(t["x"], transposed=True)
    t["w"], t["ws"], t["wt"], t["wts"] = ci8.quantize_fp8(r(n, d), block="tiles", transposed=True)
    _, _, t["stats"] = ci8.residual_norm(t["x"], t["h"], post_weight=t["post"])
    return t


CALLS = {
    "quantize_fp8": (lambda m, t, **k: m.quantize_fp8(t["x"], transposed=True, **k), dict(x="x")),
    "dequantize_fp8": (lambda m, t, **k: m.dequantize_fp8(t["q"], t["s"], **k), dict()),
    "linear_fp8": (lambda m, t, **k: m.linear_fp8(t["q"], t["w"], t["s"], t["ws"], t["bias"], activation="silu",
                                                  residual=t["res"], **k), dict(bias="bias", res="residual")),
    "linear_fp8 fp32": (lambda m, t, **k: m.linear_fp8(t["q"], t["w"], t["s"], t["ws"], t["bias"], out_dtype=torch.float32,
                                                       **k), dict(bias="bias")),
    "linear_fp8_backward": (lambda m, t, **k: m.linear_fp8_backward(t["dy"], t["qt"], t["st"], t["wt"], t["wts"], t["z"], "silu",
                                                                    **k), dict(dy="dy", z="preact")),
    "residual_norm": (lambda m, t, **k: m.residual_norm(t["x"], t["h"], t["gamma"], t["beta"], t["gate"], t["post"], **k),
                      dict(x="x", h="h", gamma="weight", beta="bias", gate="gate", post="post_weight")),
    "residual_norm_fp8": (lambda m, t, **k: m.residual_norm_fp8(t["x"], t["h"], t["gamma"], t["beta"], t["gate"], t["post"],
                                                                **k), dict(x="x", h="h")),
    "residual_norm_backward": (lambda m, t, **k: m.residual_norm_backward(t["dr"], t["x"], t["x"], t["h"], t["stats"], t["gamma"],
                                                                          t["gate"], t["post"], **k),
                               dict(dr="dr", h="h", gamma="weight", gate="gate", post="post_weight", stats="stats")),
    "clip_grad_norm": (lambda m, t, **k: (lambda outs: (m.clip_grad_norm([t["x"], t["dy"]], 1.0, out=outs, **k), *outs))(
        [torch.empty_like(t["x"]), torch.empty_like(t["dy"])]), dict(x=r"grads\[0\]", dy=r"grads\[1\]")),
}


def flat(v):
    return [u for u in (v if isinstance(v, tuple) else (v,)) if u is not None]


def same(a, b):
    return all(torch.equal(p.view(torch.uint8) if p.element_size() == 1 else p, q.view(torch.uint8) if q.element_size() == 1
                           else q) for p, q in zip(flat(a), flat(b)))


@pytest.mark.parametrize("name", list(CALLS))
def test_a_tensor_that_requires_grad_is_refused(ci8, name):
    call, operand = CALLS[name]
    want = call(ci8, operands(ci8, 6))
    for key, said in operand.items():
        t = operands(ci8, 6)
        t[key].requires_grad_()
        with pytest.raises(RuntimeError, match=f"^{said}: expects automatic differentiation"):
            call(ci8, t)
        with torch.no_grad():
            assert same(call(ci8, t), want)
        with torch.inference_mode():
            assert same(call(ci8, t), want)


@pytest.mark.parametrize("m", [5, 700])
@pytest.mark.parametrize("name", list(CALLS))
def test_operands_freed_before_the_stream_has_read_them(ci8, name, m):
    """Their memory is not handed to other work until the stream is done with the call."""
    call, _ = CALLS[name]
    want = call(ci8, operands(ci8, m))
    s = torch.cuda.Stream()
    t = operands(ci8, m)
    shapes = [(v.shape, v.dtype) for v in t.values()]
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = call(ci8, t, stream=s)
    del t
    new = [torch.empty(shape, dtype=dtype, device="cuda").view(torch.uint8).fill_(7) for shape, dtype in shapes for _ in range(2)]
    torch.cuda.current_stream().synchronize()
    s.synchronize()
    del new
    assert same(got, want)


@pytest.mark.parametrize("name", list(CALLS))
def test_a_stream_of_another_device_is_refused(ci8, name):
    other = SimpleNamespace(device=torch.device("cuda", torch.cuda.current_device() + 1))
    with pytest.raises(ValueError, match="stream: on cuda:"):
        CALLS[name][0](ci8, operands(ci8, 4), stream=other)


@pytest.mark.parametrize("m", [3, 500])
@pytest.mark.parametrize("name", list(CALLS))
def test_graph_replays(ci8, name, m):
    """Recorded and replayed on changing inputs, with eager work between the replays, two graphs in turn."""
    call, _ = CALLS[name]
    t = operands(ci8, m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            call(ci8, t)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(ci8, t))
    for i in range(3):
        for k, v in operands(ci8, m, seed=100 + i).items():
            t[k].view(torch.uint8).copy_(v.view(torch.uint8))
        for graph, out in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            got = tuple(o.clone() for o in flat(out))
            assert same(got, call(ci8, t)), i
        torch.cuda.synchronize()


def test_written_outputs_count_as_modified(ci8):
    t = operands(ci8, 40)
    for kw in (lambda e: dict(out=e), lambda e: dict(preact=e)):
        saved = torch.randn(40, 384, device="cuda").to(BF16).requires_grad_().exp()
        with torch.no_grad():
            ci8.linear_fp8(t["q"], t["w"], t["s"], t["ws"], **kw(saved.detach()))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()


@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64", "128x128d", "64x64/3"])
def test_gradients_with_every_tile(ci8, tile, monkeypatch):
    from tests.dense_reference import check
    g = torch.Generator(device="cuda").manual_seed(5)
    m, n, k = 300, 520, 264
    t = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    _, _, xt, xts = ci8.quantize_fp8(t(m, k), transposed=True)
    _, _, wt, wts = ci8.quantize_fp8(t(n, k), block="tiles", transposed=True)
    dy = t(m, n).to(BF16)
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    got = ci8.linear_fp8_backward(dy, xt, xts, wt, wts)
    for name, a, (v, e) in zip(("dx", "dw", "dbias"), got, ref.linear_backward(dy, xt, xts, wt, wts)):
        check(a, v, e, (tile, name))


# ---- together -------------------------------------------------------------------


def rounded(v, dtype):
    return v.to(dtype).double()


def q8(v, tiles=False):
    return ref.quantized(v, tiles, E4)[0]


def plain_norm(v, kind):
    mean = v.mean(-1, keepdim=True) if kind == "layer" else 0
    rstd = 1 / torch.sqrt((v - mean).square().mean(-1, keepdim=True) + 1e-5)
    return (v - mean) * rstd, rstd


def norm_gradient(c, xh, rstd, kind):
    return rstd * (c - (c.mean(-1, keepdim=True) if kind == "layer" else 0) - xh * (c * xh).mean(-1, keepdim=True))


def plain_step(stack, x, dy):
    """(y, dx, gradients of each block) of a stack in 64 bits: every tensor that the step stores rounded to its
    type, every operand of a product quantised as documented."""
    dt = x.dtype
    h, kept = None, []
    x = x.double()
    for b in stack.blocks:
        p = {k: v.double() for k, v in b.params.items()}
        hh = None
        if h is None:
            r = x
        else:
            hh, hr = plain_norm(h, b.norm)
            r = rounded(x + p["gate"] * hh * p["post"], dt)
        rh, rr = plain_norm(r, b.norm)
        y = rounded(rh * p["gamma"] + p["beta"], dt)
        z = q8(y) @ q8(b.params["w1"], True).t() + p["b1"]
        a = rounded(act(z, b.activation), dt)
        z = rounded(z, dt)
        out = rounded(q8(a) @ q8(b.params["w2"], True).t() + p["b2"], dt)
        kept.append((p, h, hh, None if h is None else hr, rh, rr, y, z, a))
        x, h = r, out
    y_out = rounded(x + h, dt)
    dr, dh, grads = dy.double(), dy.double(), []
    for b, (p, h, hh, hr, rh, rr, y, z, a) in zip(reversed(stack.blocks), reversed(kept)):
        g = {"b2": dh.sum(0), "w2": q8(dh.t().contiguous()) @ q8(a.t().contiguous()).t()}
        da = rounded(q8(dh) @ q8(b.params["w2"].t().contiguous(), True).t(), dt)
        u = da * slope(z, b.activation)
        g["b1"], g["w1"] = u.sum(0), q8(u.t().contiguous()) @ q8(y.t().contiguous()).t()
        d = rounded(q8(u) @ q8(b.params["w1"].t().contiguous(), True).t(), dt)
        g["gamma"], g["beta"] = (d * rh).sum(0), d.sum(0)
        t = dr + norm_gradient(d * p["gamma"], rh, rr, b.norm)
        if h is not None:
            g["gate"] = (t * hh * p["post"]).sum(0)
            e = t * p["gate"]
            g["post"] = (e * hh).sum(0)
            dh = rounded(norm_gradient(e * p["post"], hh, hr, b.norm), dt)
        dr = rounded(t, dt)
        grads.insert(0, g)
    return y_out, dr, grads


@pytest.mark.parametrize("rows,width,hidden,norm", [(37, 136, 520, "rms"), (300, 256, 1024, "layer"), (600, 200, 333, "rms"),
                                                    (1, 64, 128, "layer")])
def test_a_training_step(ff, rows, width, hidden, norm):
    """A value that 32-bit work leaves on the other side of a rounding differs by a step: 2^-3 of it at most in 8
    bits, 2^-7 in 16.  Few do (32-bit errors are 2^-20 of a value and less), and errors of different values are
    independent, so in the norm an output is off by a rounding or two to 16 bits, 2^-8 each, and what those change
    in the next quantisation, where one value in sixteen steps: 2^-3 / 4 of its norm for a single one, 2^-5 for
    those of a tensor."""
    stack = ff.Stack(2, width, hidden, seed=3, norm=norm)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(rows, width, generator=g, device="cuda").to(BF16)
    dy = torch.randn(rows, width, generator=g, device="cuda").to(BF16)
    y, kept = stack.forward(x)
    dx, grads = stack.backward(dy, kept)
    wy, wdx, wgrads = plain_step(stack, x, dy)
    pairs = [("y", y, wy), ("dx", dx, wdx)] + [(f"{i}.{k}", grads[i][k], v) for i, w in enumerate(wgrads) for k, v in w.items()]
    for name, got, want in pairs:
        off = float((got.double() - want).norm() / want.norm())
        assert off < 2 ** -5, (name, off)
    assert all(set(a) == set(b.params) for a, b in zip(grads, stack.blocks))

    flat_grads = [g for w in grads for g in w.values()]
    norm_want = float(torch.stack([v.double().square().sum() for v in flat_grads]).sum().sqrt())
    before = [{k: v.clone() for k, v in b.params.items()} for b in stack.blocks]
    got = stack.step(grads, 0.5, norm_want / 2)
    assert abs(float(got) - norm_want) <= 2 ** -23 * norm_want
    for b, old, g in zip(stack.blocks, before, wgrads):
        for k, v in b.params.items():
            want = old[k].double() - 0.25 * g[k]
            off = (v.double() - want).norm()
            # the gradient's own error, and a rounding of the parameter
            assert float(off) <= 2 ** -5 * 0.25 * float(g[k].norm()) + 2 ** -8 * float(want.norm()), k


def test_tokens_go_through_as_a_prompt_does(ff):
    """The form for inference quantises the unrounded norm; rows alone and in a batch take different kernels."""
    stack = ff.Stack(2, 256, 1024, seed=9)
    x = torch.randn(70, 256, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF16)
    whole, train = stack(x), stack.forward(x)[0]
    assert float((whole.double() - train.double()).norm() / train.double().norm()) < 2 ** -5
    for rows in (1, 5, 20):
        some = stack(x[:rows])
        assert float((some.double() - whole[:rows].double()).norm() / whole[:rows].double().norm()) < 2 ** -5
    assert stack(x.reshape(7, 10, 256)).shape == (7, 10, 256)


def test_the_example_runs(ff):
    losses, norms = ff.main(["--rows", "256", "--width", "128", "--hidden", "512", "--steps", "3"])
    assert len(losses) == len(norms) == 3 and all(v == v and v > 0 for v in losses + norms)
