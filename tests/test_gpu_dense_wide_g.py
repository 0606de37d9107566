"""linear_backward with g in two terms: the products' operand carries 16 or 22
bits, and small 16-bit gradients are not lost."""
import math

import pytest
import torch

from tests import dense_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def values(g, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def wanted(dy, x, w, z, act):
    """The 64-bit gradients and their bounds.  g is off by its slope's error and by
    what two roundings leave: (eps / 2)^2 of it, and in FP16 at least half of
    2^-24 of the second term, which was raised by 2^11."""
    dt, (m, n) = dy.dtype, dy.shape
    s = ref.slope(z.double(), act)
    g = dy.double() * s
    gerr = torch.zeros_like(g) if act == "relu" else (ref.SLOPE_ERR + ref.F32 * s.abs()) * dy.double().abs()
    rerr = gerr + g.abs() * (torch.finfo(dt).eps / 2) ** 2 + (2.0 ** -36 if dt == FP16 else 2.0 ** -133)
    gm, xd, wd = g.abs() + rerr, x.double(), w.double()
    dx, dw, db = g @ wd, g.t() @ xd, g.sum(0)
    ex = rerr @ wd.abs() + (2 * n + 4) * ref.F32 * (gm @ wd.abs())
    ew = rerr.t() @ xd.abs() + (2 * m + 4) * ref.F32 * (gm.t() @ xd.abs())
    eb = gerr.sum(0) + (m + 1) * ref.F32 * gm.sum(0)
    return [(v, e + ref.rounding(v.abs() + e, dt)) for v, e in ((dx, ex), (dw, ew), (db, eb))]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (3, 130, 66), (333, 129, 257), (700, 96, 64), (520, 264, 136)])
def test_wide_g(ci8, dtype, act, m, n, k):
    print(f"[gpu] linear_backward wide m={m} n={n} k={k} {dtype} {act}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(121)
    dy, x, z = values(g, m, n, dtype=dtype, scale=0.5), values(g, m, k, dtype=dtype), values(g, m, n, dtype=dtype, scale=2.0)
    w = values(g, n, k, dtype=dtype, scale=1 / math.sqrt(k))
    got = ci8.linear_backward(dy, x, w, preact=z, activation=act, wide_g=True)
    torch.cuda.synchronize()
    for name, t, (v, b) in zip(("dx", "dw", "dbias"), got, wanted(dy, x, w, z, act)):
        assert t.dtype == dtype
        ref.check(t, v, b, name)
    for i in range(3):
        part = ci8.linear_backward(dy, x, w, preact=z, activation=act, wide_g=True, need_dx=i == 0, need_dw=i == 1,
                                   need_dbias=i == 2)
        assert [p is None for p in part] == [j != i for j in range(3)] and torch.equal(part[i], got[i])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64", "128x128d", "256x256/2", "128x128/3", "64x64/5", "128x128d/2"])
def test_wide_g_on_every_tile(ci8, monkeypatch, dtype, tile):
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    print(f"[gpu] linear_backward wide tile={tile} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(122)
    m, n, k = 1400, 1329, 77
    dy, x, z = values(g, m, n, dtype=dtype), values(g, m, k, dtype=dtype), values(g, m, n, dtype=dtype)
    w = values(g, n, k, dtype=dtype, scale=0.1)
    plan = ci8.linear_backward_plan(dy, x, w, preact=z, activation="silu", wide_g=True)
    assert plan.startswith("g=written_wide launches=apart") and plan.count(f"tile={tile.split('/')[0]} ") == 2
    got = ci8.linear_backward(dy, x, w, preact=z, activation="silu", wide_g=True)
    torch.cuda.synchronize()
    for name, t, (v, b) in zip(("dx", "dw", "dbias"), got, wanted(dy, x, w, z, "silu")):
        ref.check(t, v, b, name)


def test_small_fp16_gradients(ci8):
    """dy of 2^-17 on the tail of silu: every g is below 2^-25.  One term counts them as zero, although dw, the
    sum over the rows, is well inside the type's range; two terms keep them, as dbias does."""
    m, n, k = 4096, 72, 48
    g = torch.Generator(device="cuda").manual_seed(123)
    dy = torch.full((m, n), 2.0 ** -17, dtype=FP16, device="cuda")
    z = torch.full((m, n), -9.0, dtype=FP16, device="cuda")
    x, w = values(g, m, k, dtype=FP16).abs() + 4, values(g, n, k, dtype=FP16)
    assert float((dy.double() * ref.slope(z.double(), "silu")).abs().max()) < 2.0 ** -25
    one = ci8.linear_backward(dy, x, w, preact=z, activation="silu")
    two = ci8.linear_backward(dy, x, w, preact=z, activation="silu", wide_g=True)
    want = wanted(dy, x, w, z, "silu")
    assert bool((one[1] == 0).all()) and bool((one[2] != 0).all())
    for name, t, (v, b) in zip(("dx", "dw", "dbias"), two, want):
        ref.check(t, v, b, name)
    v, b = want[1]
    assert bool((v.abs() > 8 * b).all())  # so the check above tells them from zero


def test_without_a_slope_it_is_the_same(ci8):
    g = torch.Generator(device="cuda").manual_seed(124)
    dy, x, w = values(g, 100, 64), values(g, 100, 48), values(g, 64, 48)
    for a, b in zip(ci8.linear_backward(dy, x, w, wide_g=True), ci8.linear_backward(dy, x, w)):
        assert torch.equal(a, b)
    assert ci8.linear_backward(dy[:0], x[:0], w, wide_g=True)[1].abs().max() == 0


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_nan_and_infinities(ci8, dtype):
    """They come through the first term; the second must not make NaN of an infinity."""
    g = torch.Generator(device="cuda").manual_seed(125)
    dy, x, w = values(g, 70, 72, dtype=dtype), values(g, 70, 40, dtype=dtype), values(g, 72, 40, dtype=dtype)
    z = values(g, 70, 72, dtype=dtype).abs() + 1
    x, w = x.abs() + 1, w.abs() + 1
    dy[3, 5], dy[9, 6] = math.nan, math.inf
    dx, dw, db = ci8.linear_backward(dy, x, w, preact=z, activation="gelu", wide_g=True)
    assert [i for i in range(70) if bool(torch.isnan(dx[i]).any())] == [3] and bool((dx[9] == math.inf).all())
    assert [i for i in range(72) if bool(torch.isnan(dw[i]).any())] == [5] and bool((dw[6] == math.inf).all())
    assert bool(torch.isnan(db[5])) and float(db[6]) == math.inf


def test_error_of_one_and_two_terms(ci8):
    """In the norm: the outputs' rounding alone leaves 0.0017 in BF16 and 0.00021 in FP16 (a uniform error of half a
    step over values spread evenly between powers of two); one term of g adds as much again in square."""
    g = torch.Generator(device="cuda").manual_seed(126)
    for dtype in (BF16, FP16):
        dy, x, w, z = (values(g, *s, dtype=dtype) for s in ((512, 384), (512, 320), (384, 320), (512, 384)))
        want = wanted(dy, x, w, z, "gelu_tanh")
        off = {}
        for wide in (False, True):
            got = ci8.linear_backward(dy, x, w, preact=z, activation="gelu_tanh", wide_g=wide)
            off[wide] = [float((t.double() - v).norm() / v.norm()) for t, (v, _) in zip(got[:2], want)]
        print(dtype, off)
        step = torch.finfo(dtype).eps / 2
        assert all(o < 0.5 * step for o in off[True]) and all(a < b for a, b in zip(off[True], off[False]))
