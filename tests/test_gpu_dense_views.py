"""The dense entries on views: transposed batches, gradients expanded from one
number, strided vectors, negated views -- each the same as its contiguous copy."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def same(call, *tensors, **named):
    """call on the tensors and on contiguous copies of them: the same bits."""
    plain = lambda t: t.clone(memory_format=torch.contiguous_format) if isinstance(t, torch.Tensor) else t  # noqa: E731
    a = call(*tensors, **named)
    b = call(*map(plain, tensors), **{k: plain(t) for k, t in named.items()})
    torch.cuda.synchronize()
    for p, q in zip(*((v if isinstance(v, tuple) else (v,)) for v in (a, b))):
        assert p.shape == q.shape and p.is_contiguous() and torch.equal(p, q)
    return a


def rand(*s, dtype=BF16, seed=71):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(s))
    return torch.randn(*s, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("b,s", [(3, 5), (7, 11)])
def test_transposed_batches(ci8, b, s):
    x, w, r = rand(b, s, 64).transpose(0, 1), rand(48, 64), rand(b, s, 48).transpose(0, 1)
    z, dy = rand(b, s, 48, seed=72).transpose(0, 1), rand(b, s, 48, seed=73).transpose(0, 1)
    assert same(ci8.linear, x, w, residual=r).shape == (s, b, 48)
    same(ci8.linear_backward, dy, x, w, preact=z, activation="silu")
    y, mean, rstd = same(ci8.layer_norm, x)
    assert y.shape == x.shape and mean.shape == (s, b)
    same(ci8.layer_norm_i8, x)
    same(ci8.layer_norm_backward, x.flip(-1), x, None, mean, rstd)
    t = mean.t().contiguous().t(), rstd.t().contiguous().t()  # statistics with strides of their own
    same(ci8.layer_norm_backward, x.flip(-1), x, None, *t)


@pytest.mark.parametrize("m", [5, 100])
def test_gradients_expanded_from_one_number(ci8, m):
    """What the sum of the outputs has for a gradient: strides 0 and 0."""
    one = torch.ones((), dtype=BF16, device="cuda")
    x, w, z = rand(m, 64), rand(48, 64), rand(m, 48)
    for dy in (one.expand(m, 48), one.expand(1, m, 48), rand(m, 1).expand(m, 48)):
        same(ci8.linear_backward, dy, x, w)
        same(ci8.linear_backward, dy, x, w, preact=z, activation="gelu")
    _, mean, rstd = ci8.layer_norm(x)
    same(ci8.layer_norm_backward, one.expand(m, 64), x, None, mean, rstd)
    same(ci8.linear, x, w, residual=one.expand(m, 48))


def test_strided_columns_and_vectors(ci8):
    big, v = rand(40, 192), rand(192, seed=74)
    x, w = big[:, ::3], rand(48, 64)
    same(ci8.layer_norm, x, v[::3], v[1::3])
    same(ci8.layer_norm_i8, x, v[::3], v[1::3])
    same(ci8.linear, x, w, v[::4])
    q, qw = (torch.randint(-128, 128, s, device="cuda", dtype=torch.int32).to(I8) for s in ((40, 64), (48, 64)))
    half = torch.full((1,), 0.5, device="cuda")
    same(ci8.linear, q, qw, x_scale=half.expand(40), w_scale=rand(96, dtype=FP32)[::2])


def test_negated_views(ci8):
    x = rand(9, 64, dtype=FP32)
    n = torch._neg_view(x)
    assert n.is_neg() and torch.equal(ci8.layer_norm(n)[0], ci8.layer_norm(-x)[0])
    w = rand(48, 64)
    out = torch._neg_view(rand(9, 48))
    with pytest.raises(ci8.ConvI8Error) as e:
        ci8.linear(x.to(BF16), w, out=out)
    assert e.value.name == "CONV_I8_ERR_UNSUPPORTED"


def test_outputs_keep_their_rules(ci8):
    """What is written has a contiguous last dim and leading dims that merge."""
    x, w = rand(3, 5, 64), rand(48, 64)
    for out in (rand(5, 3, 48).transpose(0, 1), rand(48, 15).t()):
        for kw in (dict(out=out), dict(preact=out)):
            with pytest.raises(ci8.ConvI8Error) as e:
                ci8.linear(x, w, **kw)
            assert e.value.name == "CONV_I8_ERR_STRIDES"


def test_views_in_a_graph(ci8):
    x, w = rand(7, 9, 64).transpose(0, 1), rand(48, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ci8.linear(ci8.layer_norm(x)[0], w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ci8.linear(ci8.layer_norm(x)[0], w)
    for i in range(3):
        x.copy_(rand(9, 7, 64, seed=80 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, ci8.linear(ci8.layer_norm(x)[0], w))
        torch.cuda.synchronize()
