"""The product of 8-bit floating point by tiles, whose results are in 16 bits: scales of every stage, split
sums and both gradients' products, on operands whose results are exact; the gradients against differences of
the product itself."""
import pytest
import torch

from tests import block_reference as ref

pytestmark = pytest.mark.gpu

E4, E5, E8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
TILES = ["256x256", "128x128", "64x64", "128x128d", "256x256/2", "128x128/3", "64x64/3", "128x128d/2"]


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def exponents(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda")


def encode(e):
    return (e + 127).to(torch.uint8).view(E8)


def by_tiles(ci8, tile, m, n, *operands):
    """That the product runs by the tile, split where its stages allow."""
    plan = ci8.linear_fp8_plan(*operands, torch.empty(m, n, dtype=torch.bfloat16))
    assert plan.startswith(f"kernel=gemm tile={tile.split('/')[0]} "), plan
    assert "/" not in tile or operands[0].shape[1] < 8 * 128 or " split=1 " not in plan, plan


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("form,tiles", [(E4, False), (E5, True)])
def test_scales_of_every_stage(ci8, tile, form, tiles, monkeypatch):
    """One value per block.  A product is a power of two from 2^-6 to 2^4 and 65 blocks add up to less than 2^11, so
    that a sum has 17 bits, which 32 hold in any order; the residual takes off what 16 bits hold of it, and what
    is left has at most eight."""
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    m, n = 260, 257
    for stages in (1, 2, 3, 4, 5, 8, 13, 15, 16, 17, 18, 31, 32, 33, 48, 65):
        g = gen(stages)
        k = 128 * stages
        x, w = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
        for b in range(stages):
            x[:, b * 128 + b * 37 % 128], w[:, b * 128 + b * 37 % 128] = 1.0, 1.0
        e, f = exponents(g, -3, 3, m, stages), exponents(g, -3, 3, ref.blocks(n) if tiles else n, stages)
        operands = (x.to(form), w.to(E4), encode(e), encode(f))
        by_tiles(ci8, tile, m, n, *operands)
        rows = f.repeat_interleave(128, 0)[:n] if tiles else f
        want = ref.pow2(e) @ ref.pow2(rows).t()
        for out in (torch.bfloat16, torch.float16):
            print("[gpu] linear_fp8", tile, form, stages, out, flush=True)
            y = ci8.linear_fp8(*operands, out_dtype=out)
            assert torch.equal(y, want.to(out)), (stages, out)
            y = ci8.linear_fp8(*operands, residual=-want.to(out), out_dtype=out)
            assert torch.equal(y.double(), want - want.to(out).double()), (stages, out)


@pytest.mark.parametrize("tile", [None] + TILES)
@pytest.mark.parametrize("dtype,form,tiles,act", [(torch.bfloat16, E4, True, "none"), (torch.float16, E5, False, "relu")])
def test_exact_gradients(ci8, tile, dtype, form, tiles, act, monkeypatch):
    """Powers of two in dy, one in a row and at most one in a column: a gradient is one product, and exact."""
    if tile:
        monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    for m, n, k in ((260, 2200, 257), (2200, 2304, 136), (40, 50, 300)):
        g = gen(m + n)
        at, rows = torch.randperm(n, generator=g, device="cuda")[:m], torch.arange(m, device="cuda")
        dy = torch.zeros(m, n, device="cuda", dtype=dtype)
        dy[rows, at] = (ref.pow2(exponents(g, -3, 4, m)) * (1 - 2 * exponents(g, 0, 2, m))).to(dtype)
        z = torch.randn(m, n, generator=g, device="cuda").to(dtype) if act == "relu" else None

        def operand(inner):
            # e4m3 numbers of 1/4 to 3.75 with their signs, in scales that 16 bits have room for
            v = torch.randint(0, 32, (k, inner), generator=g, device="cuda") + 40 + 128 * exponents(g, 0, 2, k, inner)
            return v.to(torch.uint8).view(E4), encode(exponents(g, -4, 4, ref.blocks(k) if tiles else k, ref.blocks(inner)))

        xt, xts = operand(m)
        wt, wts = operand(n)
        plan = ci8.linear_fp8_backward_plan(dy, xt, xts, wt, wts, z, act, g_dtype=form)
        print("[gpu] linear_fp8_backward", m, n, k, plan, flush=True)
        assert plan.count(f"tile={tile.split('/')[0]} ") == 2 if tile else m > 64 or "paired" in plan, plan
        dx, dw, db = ci8.linear_fp8_backward(dy, xt, xts, wt, wts, z, act, g_dtype=form)
        d = dy.double() * (z > 0) if act == "relu" else dy.double()
        live = d[rows, at][:, None]
        want = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        want[at] = live * ref.values(xt, xts).t()
        assert torch.equal(dx.double(), live * ref.values(wt, wts).t()[at]), (m, n, k, "dx")
        assert torch.equal(dw.double(), want), (m, n, k, "dw")
        assert torch.equal(db.double(), d.sum(0)), (m, n, k, "dbias")


@pytest.mark.parametrize("tile", [None, "64x64/3", "128x128/2", "256x256"])
def test_same_bits_again(ci8, tile, monkeypatch):
    if tile:
        monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    for m, n, k in ((40, 300, 5000), (600, 700, 900)):
        g = gen(m)
        x, w = (torch.randn(r, k, generator=g, device="cuda") for r in (m, n))
        q, s, qt, st = ci8.quantize_fp8(x, transposed=True)
        p, t, pt, tt = ci8.quantize_fp8(w, "tiles", transposed=True)
        dy = torch.randn(m, n, generator=g, device="cuda").to(torch.bfloat16)
        pass_ = lambda: (ci8.linear_fp8(q, p, s, t), ci8.linear_fp8(q, p, s, t, out_dtype=torch.float16),  # noqa: E731
                         *ci8.linear_fp8_backward(dy, qt, st, pt, tt))
        first = pass_()
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(pass_(), first))


@pytest.mark.parametrize("m", [5, 40])
def test_gradients_against_differences_of_the_product(ci8, m):
    """sum(dy y) of linear_fp8 in 32 bits with one value of x (w) one way and the other; both differ from 64 bits
    by their own bounds."""
    n, k = 136, 272
    g = gen(m)
    number = lambda *s: ((torch.randint(0, 64, s, generator=g, device="cuda") + 128 * exponents(g, 0, 2, *s))  # noqa: E731
                         .to(torch.uint8).view(E4))  # magnitudes up to 1.875
    ones = lambda r, c: encode(torch.zeros(r, ref.blocks(c), dtype=torch.int64, device="cuda"))  # noqa: E731
    turned = lambda t: t.view(torch.uint8).t().contiguous().view(E4)  # noqa: E731
    x, w = number(m, k), number(n, k)
    dy = torch.randint(-4, 5, (m, n), generator=g, device="cuda").to(torch.bfloat16)  # exact in 8 bits
    back = (dy, turned(x), ones(k, m), turned(w), ones(k, n))
    dx, dw, _ = ci8.linear_fp8_backward(*back)
    (_, ex), (_, ew), _ = ref.linear_backward(*back)

    def along(which, i, j):
        sums, errors = [], []
        for v in (2.0, -2.0):
            a, b = x.clone(), w.clone()
            (a, b)[which].view(torch.uint8)[i, j] = torch.tensor(v).to(E4).view(torch.uint8).item()
            args = (a, ones(m, k), b, ones(n, k))
            y = ci8.linear_fp8(a, b, args[1], args[3], out_dtype=torch.float32)
            sums.append((dy.double() * y.double()).sum())
            errors.append((dy.double().abs() * ref.linear(*args, out_dtype=torch.float32)[0][1]).sum())
        return float(sums[0] - sums[1]) / 4, float(errors[0] + errors[1]) / 4

    for i, j in ((0, 0), (m // 2, 130), (m - 1, k - 1)):
        want, error = along(0, i, j)
        assert abs(float(dx[i, j]) - want) <= error + float(ex[i, j]), (i, j)
    for i, j in ((0, 0), (70, 130), (n - 1, k - 1)):
        want, error = along(1, i, j)
        assert abs(float(dw[i, j]) - want) <= error + float(ew[i, j]), (i, j)
