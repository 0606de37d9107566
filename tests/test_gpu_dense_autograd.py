"""The dense entries beside automatic differentiation: they record nothing, so
they refuse tensors that expect it, and what they write counts as modified."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def operands():
    g = torch.Generator(device="cuda").manual_seed(61)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    return dict(x=r(6, 64), w=r(48, 64), b=r(48), res=r(6, 48), dy=r(6, 48), z=r(6, 48), gamma=r(64), beta=r(64),
                mean=torch.zeros(6, device="cuda"), rstd=torch.ones(6, device="cuda"), out=r(6, 48))


CALLS = {
    "linear": (lambda m, t: m.linear(t["x"], t["w"], t["b"], residual=t["res"], preact=t["z"], out=t["out"]),
               dict(x="x", w="w", b="bias", res="residual", z="preact", out="out")),
    "linear_backward": (lambda m, t: m.linear_backward(t["dy"], t["x"], t["w"], preact=t["z"], activation="silu"),
                        dict(dy="dy", x="x", w="w", z="preact")),
    "layer_norm": (lambda m, t: m.layer_norm(t["x"], t["gamma"], t["beta"]), dict(x="x", gamma="weight", beta="bias")),
    "layer_norm_i8": (lambda m, t: m.layer_norm_i8(t["x"], t["gamma"], t["beta"]),
                      dict(x="x", gamma="weight", beta="bias")),
    "layer_norm_backward": (lambda m, t: m.layer_norm_backward(t["x"], t["x"], t["gamma"], t["mean"], t["rstd"]),
                            dict(gamma="weight", mean="mean", rstd="rstd")),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_a_tensor_that_requires_grad_is_refused(ci8, name):
    call, operand = CALLS[name]
    for key, said in operand.items():
        t = operands()
        t[key].requires_grad_()
        with pytest.raises(RuntimeError, match=f"^{said}: expects automatic differentiation"):
            call(ci8, t)
        with torch.no_grad():
            got = call(ci8, t)
        with torch.inference_mode():
            again = call(ci8, t)
        want = call(ci8, {k: v.detach() for k, v in t.items()})
        for a, b, c in zip(*(v if isinstance(v, tuple) else (v,) for v in (got, again, want))):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_a_result_of_recorded_work_is_refused(ci8):
    t = operands()
    t["x"] = (t["x"].float().requires_grad_() * 2).to(BF16)
    with pytest.raises(RuntimeError, match="^x: expects"):
        ci8.linear(t["x"], t["w"])
    ci8.linear(t["x"].detach(), t["w"])


def test_a_forward_mode_tangent_is_refused(ci8):
    import torch.autograd.forward_ad as fwd
    t = operands()
    with fwd.dual_level():
        x = fwd.make_dual(t["x"], torch.ones_like(t["x"]))
        with pytest.raises(RuntimeError, match="expects automatic differentiation"):
            ci8.layer_norm(x)


@pytest.mark.parametrize("m", [6, 70])
def test_a_saved_tensor_that_is_overwritten_is_noticed(ci8, m):
    """exp saves its result for its gradient: written as `out` or `preact`, that gradient must not be formed from it."""
    g = torch.Generator(device="cuda").manual_seed(62)
    x, w = (torch.randn(*s, generator=g, device="cuda").to(BF16) for s in ((m, 64), (48, 64)))
    for kw in (lambda e: dict(out=e), lambda e: dict(out=e, residual=e), lambda e: dict(preact=e)):
        leaf = torch.randn(m, 48, generator=g, device="cuda").to(BF16).requires_grad_()
        saved = leaf.exp()
        version = saved._version
        with torch.no_grad():
            ci8.linear(x, w, **kw(saved.detach()))
        assert saved._version == version + 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()


def test_inside_a_function_of_ones_own(ci8):
    """The way to automatic differentiation that the documentation names."""

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            z = torch.empty(x.shape[0], w.shape[0], dtype=x.dtype, device=x.device)
            ctx.save_for_backward(x, w, z)
            return ci8.linear(x, w, b, activation="silu", preact=z)

        @staticmethod
        def backward(ctx, dy):
            x, w, z = ctx.saved_tensors
            return ci8.linear_backward(dy.contiguous(), x, w, preact=z, activation="silu")

    t = operands()
    leaves = [t[k].requires_grad_() for k in ("x", "w", "b")]
    y = Linear.apply(*leaves)
    y.backward(t["dy"])
    with torch.no_grad():
        z = torch.empty(6, 48, dtype=BF16, device="cuda")
        assert torch.equal(y, ci8.linear(*leaves, activation="silu", preact=z))
        want = ci8.linear_backward(t["dy"], leaves[0], leaves[1], preact=z, activation="silu")
    assert all(torch.equal(p.grad, q) for p, q in zip(leaves, want))
