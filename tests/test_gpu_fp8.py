"""8-bit floating point with a scale for each block of 128 on the GPU: the
quantiser bit by bit, the dense layer and its gradients against 64 bits."""
import math

import pytest
import torch

from tests import block_reference as ref
from tests.dense_reference import check

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def say(*a):
    print("[gpu]", *a, flush=True)


def wide(g, m, k, dtype=torch.float32):
    """Values over many powers of two, blocks of zeros among them."""
    x = torch.randn(m, k, generator=g, device="cuda") * torch.exp2(torch.randint(-14, 8, (m, k), generator=g, device="cuda"))
    dead = torch.rand(m, ref.blocks(k), generator=g, device="cuda") < 0.1
    return torch.where(dead.repeat_interleave(128, 1)[:, :k], 0.0, x).to(dtype)


def same_values(got, scale, want, e):
    assert scale.shape == e.shape and int((scale.view(torch.uint8).int() != e + 127).sum()) == 0
    v = ref.values(got, scale)
    wrong = ~((v == want) | (torch.isnan(v) & torch.isnan(want)))
    assert int(wrong.sum()) == 0, (v[wrong][:4].tolist(), want[wrong][:4].tolist())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("form", [E4, E5])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 128), (3, 7), (5, 129), (16, 512), (17, 513), (127, 1000), (129, 8), (300, 640)])
def test_quantize_is_exact(ci8, m, k, form, dtype):
    x = wide(gen(m * 1000 + k), m, k, DTYPES[dtype])
    for block in ("rows", "tiles"):
        tiles = block == "tiles"
        want, e = ref.quantized(x, tiles, form)
        say("quantize", m, k, form, dtype, block)
        q, s = ci8.quantize_fp8(x, block=block, dtype=form)
        same_values(q, s, want, e)
        q, s, qt, st = ci8.quantize_fp8(x, block=block, transposed=True, dtype=form)
        same_values(q, s, want, e)
        same_values(qt, st, *ref.quantized(x.t(), tiles, form))
        for t in (torch.bfloat16, torch.float32, torch.float16):
            back = ci8.dequantize_fp8(q, s, dtype=t)
            assert torch.equal(back, want.to(t)), (block, t)


def test_every_16_bit_number(ci8):
    """All bf16 and fp16 bit patterns, by themselves in blocks of their own and beside a large one."""
    for dtype in (torch.bfloat16, torch.float16):
        x = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16).view(dtype)
        for rows in (x.reshape(512, 128), x.reshape(256, 256).t().contiguous(),
                     torch.stack([x, torch.full_like(x, 3.0)], 1).reshape(-1, 128)):
            for form in (E4, E5):
                q, s = ci8.quantize_fp8(rows, dtype=form)
                same_values(q, s, *ref.quantized(rows, False, form))


def test_edges_of_the_range(ci8):
    """The largest magnitude on, below and above what the format holds; tiny and huge 32-bit values; what is not finite."""
    for form, top in ((E4, 448.0), (E5, 57344.0)):
        x = torch.zeros(12, 256, device="cuda")
        x[0, :2] = torch.tensor([top, 1.0])
        x[1, :2] = torch.tensor([math.nextafter(top, 1e9) * (1 + 2 ** -23), 1.0])
        x[2, 0], x[3, 0], x[4, 0] = 2.0 ** -149, 2.0 ** -126, 3.4e38
        x[5, 0], x[5, 1] = math.inf, 2.0
        x[6, 130], x[6, 131] = math.nan, -5.0
        x[7] = math.inf
        x[8, :3] = torch.tensor([3e38, 1e-38, -1e-30])
        x[9, 0] = -top * 2
        x[10, 0] = -0.0
        want, e = ref.quantized(x, False, form)
        assert int(e[1, 0]) == int(e[0, 0]) + 1 == 1
        q, s, qt, st = ci8.quantize_fp8(x, transposed=True, dtype=form)
        same_values(q, s, want, e)
        same_values(qt, st, *ref.quantized(x.t(), False, form))
        q, s = ci8.quantize_fp8(x, block="tiles", dtype=form)
        same_values(q, s, *ref.quantized(x, True, form))
    q = torch.zeros(1, 128, device="cuda").to(E4)
    bad = torch.full((1, 1), 255, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    assert bool(torch.isnan(ci8.dequantize_fp8(q, bad)).all())


def test_layouts(ci8):
    """Views, batches, unaligned bases and rows; memory around the outputs is not theirs to check, but rows are."""
    g = gen(5)
    x = wide(g, 40, 1000, torch.bfloat16)
    for v in (x[::2], x[:, 3:777], x[1:, 1:9], x.t(), x.reshape(4, 10, 1000), x.reshape(4, 10, 1000).transpose(0, 1),
              x[:1].expand(6, 1000), x[:, :1].expand(40, 300)):
        flat = v.reshape(-1, v.shape[-1])
        q, s, qt, st = ci8.quantize_fp8(v, transposed=True)
        assert q.shape == v.shape and s.shape == (*v.shape[:-1], ref.blocks(v.shape[-1]))
        same_values(q.reshape(flat.shape), s.reshape(flat.shape[0], -1), *ref.quantized(flat, False, E4))
        same_values(qt, st, *ref.quantized(flat.t(), False, E4))
        assert torch.equal(ci8.dequantize_fp8(q, s), ci8.dequantize_fp8(q.contiguous(), s.contiguous()))
    q, s = ci8.quantize_fp8(x)
    assert torch.equal(ci8.dequantize_fp8(q[::2], s[::2]), ci8.dequantize_fp8(q, s)[::2])
    assert torch.equal(ci8.dequantize_fp8(q[:, :256], s[:, :2]), ci8.dequantize_fp8(q, s)[:, :256])
    e = ci8.quantize_fp8(x[:0], transposed=True)
    assert e[0].shape == (0, 1000) and e[2].shape == (1000, 0)


def test_far_rows(ci8):
    """Rows further apart than 32-bit offsets reach."""
    n = (1 << 31) + 4096
    base = torch.zeros(n, dtype=torch.uint8, device="cuda")
    x = base.view(torch.bfloat16).as_strided((3, 200), ((1 << 29) - 8, 1))
    x.copy_(wide(gen(6), 3, 200, torch.bfloat16))
    q, s, qt, st = ci8.quantize_fp8(x, transposed=True)
    same_values(q, s, *ref.quantized(x, False, E4))
    same_values(qt, st, *ref.quantized(x.t(), False, E4))


def operands(g, m, n, k, xform=E4, tiles=True):
    x, e = ref.quantized(wide(g, m, k), False, xform)
    w, f = ref.quantized(wide(g, n, k) / 64, tiles, E4)
    enc = lambda v, e, t, form: ((v * ref.pow2(-ref.spread(e, v.shape, t))).float().to(form),  # noqa: E731
                                 (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu))
    return (*enc(x, e, False, xform), *enc(w, f, tiles, E4))


SHAPES = [(1, 1, 1), (1, 48, 128), (3, 130, 272), (1, 2048, 8192), (4, 100, 4096), (5, 64, 640), (16, 256, 2064),
          (17, 33, 1040), (32, 520, 4112), (33, 65, 128), (64, 64, 2176), (7, 40, 333), (130, 257, 1001), (200, 300, 5000),
          (256, 512, 16), (513, 260, 768), (9, 4100, 4112), (16, 8208, 2064), (17, 4112, 1040), (32, 4100, 640)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("xform,tiles", [(E4, True), (E4, False), (E5, True)])
def test_linear(ci8, m, n, k, xform, tiles):
    g = gen(m + n + k)
    x, xs, w, ws = operands(g, m, n, k, xform, tiles)
    say("linear_fp8", m, n, k, xform, "tiles" if tiles else "rows")
    for out, act, keep in ((torch.bfloat16, "none", False), (torch.float32, "gelu_tanh", True), (torch.float16, "silu", True)):
        b = torch.randn(n, generator=g, device="cuda").to(out)
        r = torch.randn(m, n, generator=g, device="cuda").to(out) if keep else None
        z = torch.empty(m, n, dtype=out, device="cuda") if keep else None
        y = ci8.linear_fp8(x, w, xs, ws, b, activation=act, residual=r, out_dtype=out, preact=z)
        want, wz = ref.linear(x, xs, w, ws, b, act, r, out)
        check(y, *want, ("y", m, n, k, out))
        if keep:
            check(z, *wz, ("z", m, n, k, out))


TILES = ["256x256", "128x128", "64x64", "128x128d", "256x256/3", "128x128/2", "64x64/4", "128x128d/2"]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,n,k", [(300, 270, 2500), (256, 256, 128), (70, 520, 4096), (1, 40, 2192), (512, 512, 2048)])
def test_tiles(ci8, tile, m, n, k, monkeypatch):
    """Every tile and split, with an inner dimension that ends inside a stage, a group of four and one of sixteen."""
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    g = gen(m * 7 + k)
    for xform, tiles in ((E4, True), (E5, False)):
        x, xs, w, ws = operands(g, m, n, k, xform, tiles)
        say("linear_fp8", tile, m, n, k, ci8.linear_fp8_plan(x, w, xs, ws, torch.empty(m, n, dtype=torch.bfloat16)))
        for out in (torch.bfloat16, torch.float32):
            r = torch.randn(m, n, generator=g, device="cuda").to(out)
            y = ci8.linear_fp8(x, w, xs, ws, activation="relu", residual=r, out_dtype=out)
            check(y, *ref.linear(x, xs, w, ws, None, "relu", r, out)[0], (tile, m, n, k))


@pytest.mark.parametrize("k", [128 * s for s in (1, 2, 3, 4, 5, 8, 13, 15, 16, 17, 18, 31, 32, 33, 48, 65)])
@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64", "128x128d"])
def test_scales_of_every_stage(ci8, tile, k, monkeypatch):
    """One value per block, so that a scale that belongs to another block shows: the sums are exact."""
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    g = gen(k)
    m, n = 260, 257
    x, w = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
    for b in range(k // 128):
        x[:, b * 128 + b % 128], w[:, b * 128 + b % 128] = 1.0, 1.0
    e = torch.randint(-6, 6, (m, k // 128), generator=g, device="cuda")
    f = torch.randint(-5, 5, (n, k // 128), generator=g, device="cuda")
    enc = lambda t: (t + 127).to(torch.uint8).view(torch.float8_e8m0fnu)  # noqa: E731
    y = ci8.linear_fp8(x.to(E4), w.to(E4), enc(e), enc(f), out_dtype=torch.float32)
    assert torch.equal(y.double(), torch.exp2(e.double()) @ torch.exp2(f.double()).t())
    monkeypatch.delenv("CONV_I8_DENSE_TILE")
    for rows in (1, 4, 9, 16, 25, 32):
        y = ci8.linear_fp8(x[:rows].to(E4), w.to(E4), enc(e[:rows]), enc(f), out_dtype=torch.float32)
        assert torch.equal(y.double(), torch.exp2(e[:rows].double()) @ torch.exp2(f.double()).t()), rows


@pytest.mark.parametrize("tile", [None, "256x256", "128x128", "64x64", "128x128d", "64x64/3"])
def test_small_integers_are_exact(ci8, tile, monkeypatch):
    """Integers of three bits with scales of 1 and 2: every product and sum is exact, also in what the matrix unit
    keeps of eight products, and so are the results in 16 bits where they are small."""
    if tile:
        monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    for m, n, k in ((1, 300, 2100), (20, 40, 640), (300, 270, 1040), (257, 520, 130), (64, 64, 8192)):
        g = gen(m + k)
        x, w = (torch.randint(-2, 3, (r, k), generator=g, device="cuda").float() for r in (m, n))
        enc = lambda r, c: torch.randint(127, 129, (r, c), generator=g, device="cuda").to(torch.uint8).view(torch.float8_e8m0fnu)  # noqa: E731
        xs, ws, wt = enc(m, ref.blocks(k)), enc(n, ref.blocks(k)), enc(ref.blocks(n), ref.blocks(k))
        for s in (ws, wt):
            want = ref.values(x.to(E4), xs) @ ref.values(w.to(E4), s).t()
            for form in (E4, E5):
                for out in (torch.float32, torch.bfloat16, torch.float16):
                    y = ci8.linear_fp8(x.to(form), w.to(E4), xs, s, out_dtype=out)
                    assert int((y != want.to(out)).sum()) == 0, (m, n, k, form, out)


@pytest.mark.parametrize("m", [1, 20, 150])
def test_linear_layouts(ci8, m):
    """Views of operands and scales, batches, out and residual in place."""
    g = gen(m)
    x, xs, w, ws = operands(g, m, 136, 1024, E4, False)
    want = ci8.linear_fp8(x, w, xs, ws)
    bounds = ref.linear(x, xs, w, ws)[0]
    turned = lambda t: t.view(torch.uint8).t().contiguous().t().view(t.dtype)  # noqa: E731
    pad = lambda t, c: torch.nn.functional.pad(t.view(torch.uint8), (3, c)).view(t.dtype)[:, 3:-c]  # noqa: E731
    # few rows take another kernel where an operand has to be copied: the values are then those of other sums
    for a, b, c, d in ((turned(x), w, xs, ws), (x, turned(w), xs, ws), (pad(x, 5), pad(w, 1), pad(xs, 2), pad(ws, 3))):
        check(ci8.linear_fp8(a, b, c, d), *bounds, m)
    if m > 1:
        assert torch.equal(ci8.linear_fp8(x, w, turned(xs), turned(ws)), want)
    assert torch.equal(ci8.linear_fp8(x, w, pad(xs, 2), pad(ws, 3)), want)
    assert torch.equal(ci8.linear_fp8(x.unsqueeze(0), w, xs.unsqueeze(0), ws), want.unsqueeze(0))
    if m % 2 == 0:
        b = ci8.linear_fp8(x.reshape(2, m // 2, -1), w, xs.reshape(2, m // 2, -1), ws)
        assert torch.equal(b.reshape(want.shape), want)
    r = torch.randn(m, 136, generator=g, device="cuda").to(torch.bfloat16)
    exact = ref.linear(x, xs, w, ws, out_dtype=torch.float32)[0]
    check(ci8.linear_fp8(turned(x), turned(w), xs, ws, out_dtype=torch.float32), *exact, m)
    there = ci8.linear_fp8(x, w, xs, ws, residual=r)
    out = r.clone()
    assert ci8.linear_fp8(x, w, xs, ws, residual=out, out=out).data_ptr() == out.data_ptr() and torch.equal(out, there)
    room = torch.full((m, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    ci8.linear_fp8(x, w, xs, ws, out=room[:, 5:141])
    assert torch.equal(room[:, 5:141], want) and bool((room[:, :5] == 7).all()) and bool((room[:, 141:] == 7).all())


def test_not_finite(ci8):
    """NaN in one value of x reaches its row only, NaN in w its column only, a NaN scale its row."""
    for m in (3, 70):
        x, xs, w, ws = operands(gen(m), m, 96, 640, E4, False)
        x, xs = x.clone(), xs.clone()
        x.view(torch.uint8)[1, 200] = 0x7F
        w.view(torch.uint8)[5, 7] = 0x7F
        xs.view(torch.uint8)[2, 1] = 255
        y = ci8.linear_fp8(x, w, xs, ws, out_dtype=torch.float32)
        bad = torch.zeros(m, 96, dtype=torch.bool, device="cuda")
        bad[1:3], bad[:, 5] = True, True
        assert torch.equal(torch.isnan(y), bad), m
        y = ci8.linear_fp8(x, w, xs, ws, activation="relu")
        assert torch.equal(torch.isnan(y), bad), m


def test_no_inner_dimension(ci8):
    e = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    for m in (2, 40):
        b = torch.arange(24, device="cuda").to(torch.bfloat16)
        y = ci8.linear_fp8(e(m, 0).view(E4), e(24, 0).view(E4), e(m, 0).view(torch.float8_e8m0fnu),
                           e(24, 0).view(torch.float8_e8m0fnu), b)
        assert torch.equal(y, b.expand(m, 24))


BACK = [(1, 1, 1), (1, 48, 128), (5, 33, 40), (64, 128, 256), (130, 257, 129), (333, 200, 777), (1000, 640, 72), (16, 1000, 300)]


@pytest.mark.parametrize("m,n,k", BACK)
@pytest.mark.parametrize("dtype,form,act,tiles", [("bf16", E4, "gelu_tanh", True), ("fp16", E5, "silu", False),
                                                  ("bf16", E4, "none", False), ("fp16", E4, "relu", True),
                                                  ("bf16", E5, "gelu", True)])
def test_linear_backward(ci8, m, n, k, dtype, form, act, tiles):
    g = gen(m + 3 * n + 5 * k)
    t = DTYPES[dtype]
    xt, xts, _, _ = operands(g, k, 1, m)
    _, _, wt, wts = operands(g, 1, k, n, E4, tiles)
    dy = (torch.randn(m, n, generator=g, device="cuda") * 0.1).to(t)
    z = torch.randn(m, n, generator=g, device="cuda").to(t) if act != "none" else None
    say("linear_fp8_backward", m, n, k, dtype, form, act)
    got = ci8.linear_fp8_backward(dy, xt, xts, wt, wts, preact=z, activation=act, g_dtype=form)
    want = ref.linear_backward(dy, xt, xts, wt, wts, z, act, form)
    for what, a, (v, e) in zip(("dx", "dw", "dbias"), got, want):
        check(a, v, e, (what, m, n, k))
    # each by itself, without the operand that it does not need
    assert torch.equal(ci8.linear_fp8_backward(dy, None, None, wt, wts, z, act, need_dw=False, need_dbias=False, g_dtype=form)[0], got[0])
    assert torch.equal(ci8.linear_fp8_backward(dy, xt, xts, None, None, z, act, need_dx=False, need_dbias=False, g_dtype=form)[1], got[1])
    assert torch.equal(ci8.linear_fp8_backward(dy, None, None, None, None, z, act, need_dx=False, need_dw=False)[2], got[2])


def test_backward_of_no_rows(ci8):
    u = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    _, _, wt, wts = operands(gen(1), 1, 40, 24)
    dy = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = ci8.linear_fp8_backward(dy, u(40, 0).view(E4), u(40, 0).view(torch.float8_e8m0fnu), wt, wts)
    assert dx.shape == (0, 40) and not dw.any() and not db.any() and dw.shape == (24, 40)


def test_gradients_against_differences(ci8):
    """With g exact in 8 bits (small integers), dx and dw are the derivatives of the forward product: a change of
    one value of x (w) changes sum(dy y) by that much."""
    g = gen(9)
    m, n, k = 40, 136, 272
    x, xs, w, ws = operands(g, m, n, k, E4, False)
    xd, wd = ref.values(x, xs), ref.values(w, ws)
    dy = torch.randint(-4, 5, (m, n), generator=g, device="cuda").to(torch.bfloat16)
    _, _, qt, st = ci8.quantize_fp8(xd.float(), transposed=True)
    _, _, wt, wst = ci8.quantize_fp8(wd.float(), transposed=True)
    dx, dw, _ = ci8.linear_fp8_backward(dy, qt, st, wt, wst)
    for i, j in ((0, 0), (7, 130), (39, 271)):
        up, down = xd.clone(), xd.clone()
        up[i, j] += 1.0
        down[i, j] -= 1.0
        # the formula of the forward pass, in 64 bits, at both sides
        want = float((dy.double() * ((up - down) @ ref.values(wt, wst))).sum()) / 2
        assert abs(float(dx[i, j]) - want) <= 2 ** -8 * abs(want) + 1e-4 * float(ref.values(wt, wst)[j].abs().sum())
        step = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        step[i, j] = 1.0
        want = float((dy.double() * (ref.values(qt, st).t() @ step.t())).sum())
        assert abs(float(dw[i, j]) - want) <= 2 ** -8 * abs(want) + 1e-4 * float(ref.values(qt, st)[j].abs().sum())


def test_same_bits_again(ci8):
    for m, n, k in ((1, 4096, 2048), (40, 300, 5000), (600, 700, 900)):
        x, xs, w, ws = operands(gen(2), m, n, k)
        a = ci8.linear_fp8(x, w, xs, ws, out_dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(ci8.linear_fp8(x, w, xs, ws, out_dtype=torch.float32), a)
