"""Clipping by the norm of many tensors together, on the GPU."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def make(sizes, seed=0, dtype=None, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(dtype or DTYPES[i % 3]) for i, n in enumerate(sizes)]


def reference(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def expected(grads, max_norm):
    """Values in 64 bits; off by a rounding to 32 bits and one to the type."""
    norm = reference(grads)
    return norm, [g.double() * min(1.0, max_norm / norm) for g in grads]


def close(got, want):
    info = torch.finfo(got.dtype)
    bound = want.abs() * (info.eps / 2 + 2.0 ** -23) + info.smallest_normal * info.eps
    assert bool(((got.double() - want).abs() <= bound).all()), float((got.double() - want).abs().max())


SIZES = [[1], [7], [8], [2048], [16384], [16385], [100000, 3, 16384, 0, 1, 40000], [5] * 128, [5] * 129, [300] * 500,
         [0, 0, 9], [1 << 20, 12345, 1 << 19], [(1 << 25) + 5]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_values(ci8, sizes):
    print("[gpu] clip", len(sizes), max(sizes), flush=True)
    grads = make(sizes, 3)
    norm = reference(grads)
    for limit in (norm / 3, norm * 3, 0.0):
        want_norm, want = expected(grads, limit)
        mine = [g.clone() for g in grads]
        got = ci8.clip_grad_norm(mine, limit)
        assert got.shape == () and got.dtype == torch.float32
        assert abs(float(got) - want_norm) <= 2 ** -23 * want_norm
        for a, b, g in zip(mine, want, grads):
            if limit > norm:
                assert torch.equal(a, g)
            else:
                close(a, b)
        out = [torch.full_like(g, 5) for g in grads]
        again = ci8.clip_grad_norm(grads, limit, out=out)
        assert torch.equal(again, got) and all(torch.equal(a, b) for a, b in zip(out, mine))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_factors_that_32_bits_do_not_hold(ci8, dtype):
    """Norms so far above the limit that their quotient is below 2^-126."""
    for up, limit in ((100, 2.0 ** -4), (100, 2.0 ** -40), (120, 2.0 ** 30), (120, 2.0 ** -60)):
        grads = make([1000, 9], 4, dtype, 2.0 ** up)
        norm, want = expected(grads, limit)
        got = ci8.clip_grad_norm(grads, limit)
        assert abs(float(got) - norm) <= 2 ** -23 * norm
        for a, b in zip(grads, want):
            close(a, b)


def test_shapes_and_strides(ci8):
    g = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randn(40, 60, generator=g, device="cuda")
    grads = [base.clone(), base.t().contiguous().t(), torch.randn(2, 3, 4, 5, generator=g, device="cuda").permute(3, 1, 0, 2),
             torch.randn((), generator=g, device="cuda"), torch.randn(9, generator=g, device="cuda")[1:]]
    values = [v.clone() for v in grads]
    norm = reference(grads)
    got = ci8.clip_grad_norm(grads, norm / 2)
    assert abs(float(got) - norm) <= 2 ** -23 * norm
    for a, b in zip(grads, values):
        close(a, b.double() / 2)


def test_out_with_other_strides_along_dims_of_one(ci8):
    """They say nothing about where the values lie: a gradient of a column as its transpose leaves it."""
    base = torch.arange(1.0, 41, device="cuda")
    for g, out in ((base.reshape(1, 40).t(), torch.zeros(40, 1, device="cuda")),
                   (base.as_strided((1, 5, 8), (3, 8, 1)), torch.zeros(1, 5, 8, device="cuda")),
                   (base[:1].as_strided((1, 1), (7, 9)), torch.zeros(1, 1, device="cuda"))):
        norm = reference([g])
        ci8.clip_grad_norm([g], norm / 2, out=[out])
        close(out, g.double() / 2)


def test_refusals(ci8):
    x = torch.ones(8, 8, device="cuda")
    for grads, out, status in (([x[:, ::2]], None, "STRIDES"), ([x[:, :4]], None, "STRIDES"), ([x[:1].expand(4, 8)], None, "STRIDES"),
                               ([x, x], None, "PARAM"), ([x, x[2:4]], None, "PARAM"), ([x], [x.t()], "STRIDES"),
                               ([x], [x.clone(), x.clone()], "OUT_DIMS"), ([x], [x.to(torch.bfloat16)], "DTYPE"),
                               ([x.to(torch.int32)], None, "DTYPE"), ([x.double()], None, "DTYPE"), ([x], [torch.ones(64, device="cuda")], "OUT_DIMS")):
        with pytest.raises(ci8.ConvI8Error) as e:
            ci8.clip_grad_norm(grads, 1.0, out=out)
        assert e.value.name == "CONV_I8_ERR_" + status
    for limit in (-1.0, math.nan):
        with pytest.raises(ci8.ConvI8Error):
            ci8.clip_grad_norm([x], limit)
    assert bool((x == 1).all())
    p = torch.ones(4, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match=r"grads\[1\]: expects automatic differentiation"):
        ci8.clip_grad_norm([x, p], 1.0)
    with torch.no_grad():
        ci8.clip_grad_norm([x, p], 100.0)


def next_to_the_middle(dtype):
    """(value, factor) pairs whose product is a little above the middle of two numbers of `dtype`, by more than a
    rounding to 32 bits takes off, where a factor and a product of 32 bits give the middle or less."""
    bits = {torch.bfloat16: 8, torch.float16: 11}[dtype]
    found = []
    for i in range(1, 9000, 2):
        value = 1.0 + (i % 2 ** (bits - 1)) * 2.0 ** (1 - bits)
        middle = 0.5 + (2 * ((7 * i) % 2 ** (bits - 2)) + 0.5) * 2.0 ** -bits  # above an even number
        factor = middle * (1 + 0.8 * 2.0 ** -23) / value
        near = torch.tensor(value) * torch.tensor(factor, dtype=torch.float64).float()
        if value * factor > middle >= float(near) and float(torch.tensor(value * factor, dtype=torch.float64).float()) > middle:
            found.append((value, factor))
    return found


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_products_next_to_the_middle(ci8, dtype):
    """16-bit values times the factor in 64 bits: the sum of squares is exact here, and so the factor is the same."""
    pairs = next_to_the_middle(dtype)
    assert len(pairs) > 20
    for value, factor in pairs[::max(1, len(pairs) // 20)]:
        g = [torch.full((9,), value, device="cuda", dtype=dtype), torch.full((40,), -value, device="cuda", dtype=dtype)]
        limit = factor * (7 * value)  # 49 values: the norm is exact
        want = [(v.double() * (limit / (7 * value))).float().to(dtype) for v in g]
        assert float(ci8.clip_grad_norm(g, limit)) == 7 * value
        assert all(torch.equal(a, b) for a, b in zip(g, want)), (value, factor)


def test_factors_far_below_32_bits(ci8):
    """Factors of 2^-130 to 2^-240, whose products with BF16 values are still numbers of that type: the same rounding."""
    for up, limit in ((100, 1.7 * 2.0 ** -30), (120, 1.3 * 2.0 ** -70), (120, 1.9 * 2.0 ** -100), (126, 1.1 * 2.0 ** -114)):
        g = [(torch.arange(1, 129, device="cuda") / 128 * 2.0 ** up).to(torch.bfloat16)]
        norm = math.sqrt(float(g[0].double().square().sum()))
        want = (g[0].double() * (limit / norm)).to(torch.bfloat16)
        ci8.clip_grad_norm(g, limit)
        assert bool(want.any()) and torch.equal(g[0], want), (up, limit)


def test_norms_that_32_bits_do_not_hold(ci8):
    """Finite values whose norm reads as infinity are scaled by it all the same, in place and into `out`; only values
    that are not finite stay as they are."""
    for dtype in (torch.bfloat16, torch.float32):
        grads = [torch.full((5000,), 3e38, device="cuda", dtype=dtype), make([33], 2, dtype)[0]]
        norm, want = expected(grads, 8.0)
        assert norm > torch.finfo(torch.float32).max
        out = [torch.empty_like(g) for g in grads]
        assert float(ci8.clip_grad_norm(grads, 8.0, out=out)) == math.inf
        assert float(ci8.clip_grad_norm(grads, 8.0)) == math.inf
        for a, b, c in zip(grads, out, want):
            assert torch.equal(a, b)
            close(a, c)


def test_range(ci8):
    """Squares that 32 bits cannot hold; norms that are not finite change nothing; zeros."""
    big = [torch.full((1000,), 3e38, device="cuda"), torch.full((10,), 1e-38, device="cuda")]
    small = [torch.full((50000,), 1e-30, device="cuda")]
    for grads in ([b.clone() for b in big[:1]], small):
        norm = reference(grads)
        got = float(ci8.clip_grad_norm(grads, norm / 1e3))
        assert got == float(torch.tensor(norm, dtype=torch.float64).float()) or abs(got - norm) <= 2 ** -23 * norm
        assert abs(reference(grads) - norm / 1e3) <= 2 ** -22 * norm / 1e3
    for bad in (math.inf, math.nan, -math.inf):
        grads = make([100, 200], 5)
        grads[1][7] = bad
        before = [g.clone() for g in grads]
        got = float(ci8.clip_grad_norm(grads, 0.1))
        assert not math.isfinite(got)
        assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip(grads, before))
        out = [torch.zeros_like(g) for g in grads]
        ci8.clip_grad_norm(grads, 0.1, out=out)
        assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip(out, before))
    zeros = [torch.zeros(5, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(ci8.clip_grad_norm(zeros, 0.0)) == 0.0 and not zeros[0].any()
    x = make([64], 1, torch.float32)
    y = x[0].clone()
    ci8.clip_grad_norm(x, math.inf)
    assert torch.equal(x[0], y)


def test_written_tensors_count_as_modified(ci8):
    leaf = torch.ones(8, device="cuda", requires_grad=True)
    saved = leaf.exp()
    ci8.clip_grad_norm([saved.detach()], 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.sum().backward()


def test_same_bits_again(ci8):
    grads = make([1 << 20, 70000, 3], 9, torch.bfloat16)
    out = [torch.empty_like(g) for g in grads]
    first = ci8.clip_grad_norm(grads, 1.0, out=out)
    kept = [o.clone() for o in out]
    for _ in range(3):
        assert torch.equal(ci8.clip_grad_norm(grads, 1.0, out=out), first) and all(torch.equal(a, b) for a, b in zip(out, kept))
