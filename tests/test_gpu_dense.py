"""The dense layer and layer norm, forward and backward, on the GPU against
their 64-bit forms, with bounds that count 32-bit and output roundings.

Operands sit in larger buffers whose gaps hold NaN (or the int8 extreme), so
that a value read from outside an operand shows, and outputs in buffers whose
gaps hold a sentinel that has to survive."""
import math

import pytest
import torch

from tests import dense_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def values(g, *shape, dtype=BF16, scale=1.0):
    if dtype == I8:
        return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(I8)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def embed(t, pitch=0, offset=0, cols_major=False):
    """The matrix in a larger buffer: `pitch` more elements per row, the first
    element `offset` elements into it; everything else NaN (-128 for int8)."""
    if cols_major:
        return embed(t.t(), pitch, offset).t()
    r, c = t.shape
    fill = -128 if t.dtype == I8 else math.nan
    buf = torch.full((offset + (r + 1) * (c + pitch) + 64,), fill, dtype=t.dtype, device=t.device)
    v = buf.as_strided((r, c), (c + pitch, 1), offset)
    v.copy_(t)
    return v


class Out:
    """An output matrix inside a buffer of sentinels."""

    def __init__(self, r, c, dtype, pitch=0, offset=0):
        self.buf = torch.full((offset + (r + 1) * (c + pitch) + 64,), -77.0, dtype=dtype, device="cuda")
        self.t = self.buf.as_strided((r, c), (c + pitch, 1), offset)
        self.where = torch.zeros(self.buf.shape, dtype=torch.bool, device="cuda")
        self.where.as_strided((r, c), (c + pitch, 1), offset).fill_(True)

    def check_gaps(self):
        assert bool((self.buf[~self.where] == -77.0).all()), "written outside the output"


def run_linear(ci8, m, n, k, dtype, act="none", residual=False, keep=False, bias=True, out_dtype=None, seed=1,
               x_layout={}, w_layout={}, out_layout={}, scales=True):
    print(f"[gpu] linear m={m} n={n} k={k} {dtype} act={act} residual={residual} keep={keep} out={out_dtype} "
          f"x={x_layout} w={w_layout} out={out_layout}", flush=True)
    g = gen(seed)
    out_dtype = out_dtype or (BF16 if dtype == I8 else dtype)
    x = embed(values(g, m, k, dtype=dtype), **x_layout)
    w = embed(values(g, n, k, dtype=dtype, scale=1 / math.sqrt(max(k, 1))), **w_layout)
    b = values(g, n, dtype=out_dtype) if bias else None
    r = embed(values(g, m, n, dtype=out_dtype), **out_layout) if residual else None
    xs = ws = None
    if dtype == I8 and scales:
        xs = (torch.rand(m, generator=g, device="cuda") + 0.5) / 64
        ws = (torch.rand(n, generator=g, device="cuda") + 0.5) / (64 * math.sqrt(max(k, 1)))
    o, z = Out(m, n, out_dtype, **out_layout), Out(m, n, out_dtype, **out_layout)
    y = ci8.linear(x, w, b, activation=act, residual=r, x_scale=xs, w_scale=ws, out=o.t,
                   preact=z.t if keep else None)
    torch.cuda.synchronize()
    assert y is o.t
    (yv, yb), (zv, zb) = ref.linear(x, w, b, act, r, xs, ws, out_dtype)
    ref.check(y, yv, yb, "y")
    o.check_gaps()
    if keep:
        ref.check(z.t, zv, zb, "z")
    z.check_gaps()


# rows of x from one to past the few-rows kernel, odd and aligned widths
@pytest.mark.parametrize("dtype", [BF16, FP16, I8])
@pytest.mark.parametrize("m", [1, 2, 7, 16, 17, 31, 32])
@pytest.mark.parametrize("n,k", [(64, 64), (1, 1), (33, 130), (257, 1024), (40, 4096 + 16), (16, 4099)])
def test_linear_few_rows(ci8, dtype, m, n, k):
    act = ACTS[(m + n) % 5]
    run_linear(ci8, m, n, k, dtype, act=act, residual=m % 2 == 1, keep=n % 2 == 1)


@pytest.mark.parametrize("dtype", [BF16, FP16, I8])
@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64"])
@pytest.mark.parametrize("m,n,k", [(256, 256, 64), (300, 200, 160), (65, 513, 1056), (1, 8, 32), (513, 264, 96)])
def test_linear_tiles(ci8, monkeypatch, dtype, tile, m, n, k):
    """Every tile at full, partial and near-empty tiles, odd and even stage counts."""
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    run_linear(ci8, m, n, k, dtype, act=ACTS[(m + k // 32) % 5], residual=m % 2 == 0, keep=True)


@pytest.mark.parametrize("dtype", [BF16, FP16, I8])
@pytest.mark.parametrize("tile", ["256x256/3", "128x128/2", "128x128/8", "64x64/5"])
@pytest.mark.parametrize("m,n,k", [(130, 100, 4096), (33, 257, 2080)])
def test_linear_split(ci8, monkeypatch, dtype, tile, m, n, k):
    """The inner dimension split over workgroups, partial sums joined in order."""
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    run_linear(ci8, m, n, k, dtype, act="gelu_tanh", residual=True, keep=True)


@pytest.mark.parametrize("dtype", [BF16, FP16, I8])
@pytest.mark.parametrize("m,n,k", [(33, 1, 1), (40, 3, 7), (331, 101, 283), (97, 1001, 77), (64, 72, 8), (50, 50, 0),
                                   (5, 50, 0)])
def test_linear_odd_sizes(ci8, dtype, m, n, k):
    run_linear(ci8, m, n, k, dtype, act="silu", residual=True, keep=True)


@pytest.mark.parametrize("dtype", [BF16, I8])
@pytest.mark.parametrize("m", [3, 96])
@pytest.mark.parametrize("layouts", [
    dict(x_layout=dict(pitch=16), w_layout=dict(pitch=32), out_layout=dict(pitch=8)),
    dict(x_layout=dict(pitch=3), w_layout=dict(pitch=1), out_layout=dict(pitch=5)),
    dict(x_layout=dict(offset=1), w_layout=dict(offset=3), out_layout=dict(offset=1)),
    dict(x_layout=dict(cols_major=True)),
    dict(w_layout=dict(cols_major=True)),
    dict(x_layout=dict(cols_major=True, pitch=8), w_layout=dict(cols_major=True, pitch=8)),
    dict(w_layout=dict(cols_major=True, pitch=3, offset=1)),
])
def test_linear_layouts(ci8, dtype, m, layouts):
    run_linear(ci8, m, 136, 160, dtype, act="relu", residual=True, keep=True, **layouts)


@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64"])
@pytest.mark.parametrize("m,n,k", [(300, 520, 200), (70, 72, 31)])
def test_linear_transposed_weights_in_place(ci8, monkeypatch, tile, m, n, k):
    """A [K, N] weight read through its transposed view, without a copy."""
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    w = torch.empty(k, n, dtype=BF16, device="cuda").t()
    assert "b=cols " in ci8.linear_plan(torch.empty(m, k, dtype=BF16), w, torch.empty(m, n, dtype=BF16)) + " "
    run_linear(ci8, m, n, k, BF16, w_layout=dict(cols_major=True))


def test_linear_broadcast_and_strided_operands(ci8):
    """Rows repeated by a zero stride, and both strides other than one."""
    g = gen(3)
    row = values(g, 1, 96)
    w = values(g, 40, 96)
    for m in (4, 64):
        x = row.expand(m, 96)
        (v, b), _ = ref.linear(x, w, out_dtype=BF16)
        ref.check(ci8.linear(x, w), v, b, f"expanded rows {m}")
        big = values(g, 2 * m, 3 * 96)
        x = big[::2, ::3]
        ws = values(g, 80, 192)[::2, ::2]
        (v, b), _ = ref.linear(x, ws, out_dtype=BF16)
        ref.check(ci8.linear(x, ws), v, b, f"strided {m}")


@pytest.mark.parametrize("dtype,out", [(BF16, FP32), (FP16, FP32), (I8, FP16), (I8, FP32), (I8, BF16)])
@pytest.mark.parametrize("m", [5, 70])
def test_linear_output_types(ci8, dtype, out, m):
    run_linear(ci8, m, 77, 64, dtype, act="gelu", residual=True, keep=True, out_dtype=out)
    run_linear(ci8, m, 77, 64, dtype, bias=False, out_dtype=out, scales=False)


def test_linear_int8_extremes(ci8):
    """The longest exact reduction of the extreme values, and one more refused."""
    k = 131071
    for m in (2, 40):
        x = torch.full((m, k), -128, dtype=I8, device="cuda")
        w = torch.full((24, k), -128, dtype=I8, device="cuda")
        y = ci8.linear(x, w, out_dtype=FP32)
        assert bool((y.double() == float(torch.tensor(128.0 * 128 * k, dtype=FP32))).all())
    x = torch.zeros((2, k + 1), dtype=I8, device="cuda")
    with pytest.raises(ci8.ConvI8Error) as e:
        ci8.linear(x, x)
    assert e.value.name == "CONV_I8_ERR_RANGE"


@pytest.mark.parametrize("m", [3, 80])
@pytest.mark.parametrize("act", ACTS)
def test_linear_nonfinite(ci8, m, act):
    """NaN and infinities reach their own row (of x) and column (of w) and no other."""
    g = gen(5)
    x, w = values(g, m, 72), values(g, 48, 72)
    x[1, 70] = math.nan
    w[7, 3] = math.nan
    y, z = ci8.linear(x, w, activation=act), torch.empty(m, 48, dtype=BF16, device="cuda")
    bad = torch.zeros(m, 48, dtype=torch.bool, device="cuda")
    bad[1] = True
    bad[:, 7] = True
    assert bool((torch.isnan(y) == bad).all())
    x[1, 70], w[7, 3] = 0, 0
    x[2, 5] = math.inf
    w[:, 5] = w[:, 5].abs() + 1
    y = ci8.linear(x, w, activation=act, preact=z)
    assert bool((z[2] == math.inf).all()) and bool((y[2] == math.inf).all())
    keep = [i for i in range(m) if i != 2]
    (v, b), _ = ref.linear(x[keep], w, activation=act, out_dtype=BF16)
    ref.check(y[keep], v, b, "other rows")


def test_linear_batched_and_default_outputs(ci8):
    g = gen(6)
    x, w = values(g, 3, 5, 64), values(g, 32, 64)
    r = values(g, 3, 5, 32)
    y = ci8.linear(x, w, residual=r)
    assert y.shape == (3, 5, 32) and y.dtype == BF16
    (v, b), _ = ref.linear(x.view(15, 64), w, residual=r.view(15, 32), out_dtype=BF16)
    ref.check(y.view(15, 32), v, b, "batched")
    one = ci8.linear(x[0, 0], w)
    assert one.shape == (32,)
    q = ci8.linear(values(g, 2, 64, dtype=I8), values(g, 8, 64, dtype=I8), x_scale=torch.ones(2, device="cuda"))
    assert q.dtype == BF16
    for shape in ((0, 64), (4, 0, 64)):
        assert ci8.linear(torch.empty(shape, dtype=BF16, device="cuda"), w).shape == (*shape[:-1], 32)
    assert ci8.linear(x, torch.empty(0, 64, dtype=BF16, device="cuda")).shape == (3, 5, 0)


@pytest.mark.parametrize("m", [4, 200])
def test_linear_in_place_residual(ci8, m):
    g = gen(7)
    x, w, h = values(g, m, 96), values(g, 104, 96, scale=0.1), values(g, m, 104)
    (v, b), _ = ref.linear(x, w, activation="silu", residual=h.clone(), out_dtype=BF16)
    y = ci8.linear(x, w, activation="silu", residual=h, out=h)
    assert y is h
    ref.check(h, v, b, "in place")


def run_backward(ci8, m, n, k, dtype, act="none", seed=1, dy_layout={}, x_layout={}, w_layout={}, z_layout={}):
    print(f"[gpu] linear_backward m={m} n={n} k={k} {dtype} act={act} dy={dy_layout} x={x_layout} w={w_layout}", flush=True)
    g = gen(seed)
    dy = embed(values(g, m, n, dtype=dtype, scale=0.5), **dy_layout)
    x = embed(values(g, m, k, dtype=dtype), **x_layout)
    w = embed(values(g, n, k, dtype=dtype, scale=1 / math.sqrt(max(k, 1))), **w_layout)
    z = embed(values(g, m, n, dtype=dtype, scale=2.0), **z_layout) if act != "none" else None
    got = ci8.linear_backward(dy, x, w, preact=z, activation=act)
    torch.cuda.synchronize()
    for name, t, (v, b) in zip(("dx", "dw", "dbias"), got, ref.linear_backward(dy, x, w, z, act)):
        assert t.dtype == dtype
        ref.check(t, v, b, name)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 64, 72), (3, 130, 66), (40, 520, 264), (333, 129, 257), (700, 96, 64)])
def test_backward(ci8, dtype, act, m, n, k):
    run_backward(ci8, m, n, k, dtype, act)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64", "256x256/2", "128x128/4", "128x128/3", "64x64/7"])
@pytest.mark.parametrize("m,n,k", [(520, 264, 300), (289, 1040, 96)])
def test_backward_tiles(ci8, monkeypatch, dtype, tile, m, n, k):
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    run_backward(ci8, m, n, k, dtype, "gelu_tanh")


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("layouts", [
    dict(dy_layout=dict(pitch=8), x_layout=dict(pitch=16), w_layout=dict(pitch=8), z_layout=dict(pitch=24)),
    dict(dy_layout=dict(pitch=1), x_layout=dict(pitch=3), w_layout=dict(pitch=5), z_layout=dict(pitch=7)),
    dict(dy_layout=dict(offset=1), x_layout=dict(offset=3), w_layout=dict(offset=5), z_layout=dict(offset=1)),
    dict(x_layout=dict(cols_major=True), w_layout=dict(cols_major=True)),
])
def test_backward_layouts(ci8, act, layouts):
    run_backward(ci8, 144, 136, 120, BF16, act, **layouts)


def test_backward_broadcast_gradient(ci8):
    """A gradient that repeats one row (zero stride)."""
    g = gen(9)
    dy, x, w = values(g, 1, 64).expand(50, 64), values(g, 50, 48), values(g, 64, 48)
    for t, (v, b) in zip(ci8.linear_backward(dy, x, w), ref.linear_backward(dy, x, w)):
        ref.check(t, v, b, "broadcast")


def test_backward_parts_and_empty(ci8):
    g = gen(10)
    dy, x, w, z = values(g, 40, 64), values(g, 2, 20, 48), values(g, 64, 48), values(g, 2, 20, 64)
    full = ci8.linear_backward(dy.view(2, 20, 64), x, w, preact=z, activation="gelu")
    assert full[0].shape == x.shape
    for i in range(3):
        need = dict(need_dx=i == 0, need_dw=i == 1, need_dbias=i == 2)
        part = ci8.linear_backward(dy.view(2, 20, 64), x, w, preact=z, activation="gelu", **need)
        assert [p is None for p in part] == [j != i for j in range(3)]
        assert torch.equal(part[i], full[i])
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    dx, dw, db = ci8.linear_backward(e(0, 64), e(0, 48), w)
    assert dx.shape == (0, 48) and bool((dw == 0).all()) and bool((db == 0).all())
    dx, dw, db = ci8.linear_backward(e(5, 0), x[0, :5].contiguous(), e(0, 48))
    assert bool((dx == 0).all()) and dw.shape == (0, 48) and db.shape == (0,)


def test_backward_nan_stays_in_its_row_and_column(ci8):
    g = gen(11)
    dy, x, w = values(g, 70, 72), values(g, 70, 40), values(g, 72, 40)
    dy[3, 5] = math.nan
    dx, dw, db = ci8.linear_backward(dy, x, w)
    assert [bool(torch.isnan(dx[i]).any()) for i in range(70)] == [i == 3 for i in range(70)]
    assert [bool(torch.isnan(dw[i]).any()) for i in range(72)] == [i == 5 for i in range(72)]
    assert [bool(v) for v in torch.isnan(db)] == [i == 5 for i in range(72)]


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh"])
def test_backward_matches_differences(ci8, act):
    """Along a random direction, the gradients' inner product with it is the
    central difference of the loss sum(dy * linear(x, w, b)) in 64 bits.  The
    kernel's rounding of its outputs bounds the difference: each entry of a
    gradient is off by at most its bound, plus h^2 of the third derivative
    (below 10 |v|^3 here, relu: its kink, avoided by values away from 0)."""
    g = gen(12)
    m, n, k = 24, 40, 32
    x, w, b, dy = (values(g, *s, dtype=FP16) for s in ((m, k), (n, k), (n,), (m, n)))
    w = (w.double() / 8).to(FP16)
    z = x.double() @ w.double().t() + b.double()
    zh = z.to(FP16)
    got = ci8.linear_backward(dy, x, w, preact=zh, activation=act)
    bounds = ref.linear_backward(dy, x, w, zh, act)
    h = 1e-4
    for i, base in enumerate((x, w, b)):
        v = torch.randn(*base.shape, generator=g, device="cuda", dtype=torch.float64)
        v = v / v.abs().max()

        def loss(s):
            p = [t.double() for t in (x, w, b)]
            p[i] = p[i] + s * v
            zz = p[0] @ p[1].t() + p[2]
            # the kernel's slope is taken at the rounded z, so the difference is too
            lin = zz - z + zh.double()
            if act == "relu":  # no value changes its sign between the two sides
                return (dy.double() * torch.where(zh.double() > 0, lin, torch.zeros_like(lin))).sum()
            return (dy.double() * ref.act(lin, act)).sum()

        diff = float((loss(h) - loss(-h)) / (2 * h))
        mine = float((got[i].double() * v).sum())
        tol = float((bounds[i][1] * v.abs()).sum()) + 1e-3 * h * m * n + 1e-6
        assert abs(diff - mine) <= tol, (act, i, diff, mine, tol)


def run_norm(ci8, m, d, dtype, seed=1, weight=True, bias=True, eps=1e-5, layout={}, shift=1.0, scale=1.5):
    print(f"[gpu] layer_norm m={m} d={d} {dtype} weight={weight} bias={bias} eps={eps} {layout}", flush=True)
    g = gen(seed)
    x = embed((torch.randn(m, d, generator=g, device="cuda") * scale + shift).to(dtype), **layout)
    w = values(g, d, dtype=dtype) if weight else None
    b = values(g, d, dtype=dtype) if bias else None
    want = ref.layer_norm(x, w, b, eps)
    y, mean, rstd = ci8.layer_norm(x, w, b, eps=eps)
    torch.cuda.synchronize()
    assert y.dtype == dtype and mean.dtype == rstd.dtype == FP32
    ref.check(mean, *want["mean"], "mean")
    ref.check(rstd, *want["rstd"], "rstd")
    v, e = want["y"]
    ref.check(y, v, e + ref.rounding(v.abs() + e, dtype), "y")
    q, s = ci8.layer_norm_i8(x, w, b, eps=eps)
    torch.cuda.synchronize()
    assert q.dtype == I8 and s.dtype == FP32
    top = v.abs().amax(1)
    es = e.amax(1) / 127 + 2 * ref.F32 * (top / 127)
    ref.check(s, top / 127, es, "scale")
    # half a step of the scale, and what y and the scale are off (the scale's error times |q| <= 127)
    ref.check(q.double() * s.double()[:, None], v,
              0.5 * (top / 127 + es)[:, None] * (1 + 2 ** -10) + e + 127 * es[:, None], "q * scale")
    assert bool((q.abs().amax(1) == 127).all()) or bool((top == 0).any())


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("m,d", [(1, 1), (3, 2), (5, 7), (2, 64), (4, 513), (7, 1000), (3, 2048), (2, 2049), (5, 4096),
                                 (3, 5000), (2, 8192), (3, 10001), (2, 16384), (3, 20000), (2, 65536), (2, 65537), (1, 70001),
                                 (1100, 200), (1100, 777), (1100, 1531), (1030, 2048)])
def test_norm(ci8, dtype, m, d):
    run_norm(ci8, m, d, dtype, weight=d % 3 != 0, bias=d % 5 != 0)


@pytest.mark.parametrize("layout", [dict(pitch=8), dict(pitch=1), dict(offset=3), dict(pitch=5, offset=1)])
@pytest.mark.parametrize("d", [96, 2000, 9000, 66000])
def test_norm_layouts(ci8, layout, d):
    run_norm(ci8, 5, d, BF16, layout=layout)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_norm_far_mean_and_eps(ci8, dtype):
    """A mean far above the spread (two passes over registers keep the variance), and eps of 0 and 1."""
    run_norm(ci8, 6, 3000, dtype, shift=100.0, scale=1.0)
    run_norm(ci8, 6, 300, dtype, eps=0.0)
    run_norm(ci8, 6, 300, dtype, eps=1.0)


def test_norm_constant_and_nonfinite_rows(ci8):
    """A constant row gives the bias; without one its int8 row is zero with scale 0.  NaN stays in its row."""
    for d in (8, 600, 3000, 70000):
        x = torch.ones(4, d, dtype=BF16, device="cuda")
        b = torch.full((d,), 0.5, dtype=BF16, device="cuda")
        y, _, _ = ci8.layer_norm(x, None, b)
        assert bool((y == 0.5).all())
        q, s = ci8.layer_norm_i8(x)
        assert bool((q == 0).all()) and bool((s == 0).all())
        x = torch.randn(4, d, device="cuda").to(BF16)
        x[1, d // 2] = math.nan
        x[2, 0] = math.inf
        y, mean, rstd = ci8.layer_norm(x)
        assert bool(torch.isnan(y[1:3]).all()) and not bool(torch.isnan(y[[0, 3]]).any())
        q, s = ci8.layer_norm_i8(x)
        assert [bool(v) for v in torch.isnan(s)] == [False, True, True, False]


def test_norm_batched_and_empty(ci8):
    g = gen(13)
    x = values(g, 3, 4, 96)
    y, mean, rstd = ci8.layer_norm(x)
    assert y.shape == x.shape and mean.shape == rstd.shape == (3, 4)
    flat = ci8.layer_norm(x.view(12, 96))
    assert torch.equal(y.view(12, 96), flat[0]) and torch.equal(mean.view(12), flat[1])
    q, s = ci8.layer_norm_i8(x)
    assert q.shape == x.shape and s.shape == (3, 4)
    dx, dw, db = ci8.layer_norm_backward(x, x, None, mean, rstd)
    assert dx.shape == x.shape
    e = torch.empty(0, 96, dtype=BF16, device="cuda")
    y, mean, rstd = ci8.layer_norm(e)
    assert y.shape == (0, 96) and mean.shape == (0,)
    dx, dw, db = ci8.layer_norm_backward(e, e, None, mean, rstd)
    assert dx.shape == (0, 96) and bool((dw == 0).all()) and bool((db == 0).all())


def run_norm_backward(ci8, m, d, dtype, seed=1, weight=True, layout={}):
    print(f"[gpu] layer_norm_backward m={m} d={d} {dtype} weight={weight} {layout}", flush=True)
    g = gen(seed)
    x = embed((torch.randn(m, d, generator=g, device="cuda") * 1.5 + 1).to(dtype), **layout)
    dy = embed(values(g, m, d, dtype=dtype), **layout)
    w = values(g, d, dtype=dtype) if weight else None
    mean = x.double().mean(1).float()
    rstd = (1 / torch.sqrt(x.double().var(1, correction=0) + 1e-5)).float()
    got = ci8.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    for name, t, (v, b) in zip(("dx", "dweight", "dbias"), got, ref.layer_norm_backward(dy, x, w, mean, rstd)):
        assert t.dtype == dtype
        ref.check(t, v, b, name)
    alone = ci8.layer_norm_backward(dy, x, w, mean, rstd, need_params=False)
    assert torch.equal(alone[0], got[0]) and alone[1] is None and alone[2] is None


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("m,d", [(1, 1), (2, 3), (5, 64), (3, 512), (9, 513), (2, 2048), (7, 2049), (3, 4096), (5, 8000),
                                 (3, 8193), (2, 16384), (3, 16385), (2, 33333), (70, 20000), (2500, 96), (4000, 600),
                                 (1003, 1537), (2200, 2100)])
def test_norm_backward(ci8, dtype, m, d):
    run_norm_backward(ci8, m, d, dtype, weight=d % 3 != 0)


@pytest.mark.parametrize("layout", [dict(pitch=8), dict(pitch=3), dict(offset=1)])
@pytest.mark.parametrize("d", [100, 1030, 9000, 17000])
def test_norm_backward_layouts(ci8, layout, d):
    run_norm_backward(ci8, 21, d, BF16, layout=layout)


def test_norm_backward_matches_differences(ci8):
    """The gradients' inner product with a random direction against the
    central difference of sum(dy * layer_norm(x)) in 64 bits; what is left is
    the gradients' own rounding and h^2 of the third derivative."""
    g = gen(14)
    m, d, h = 6, 50, 1e-4
    x, w, b, dy = (torch.randn(*s, generator=g, device="cuda") for s in ((m, d), (d,), (d,), (m, d)))
    y, mean, rstd = ci8.layer_norm(x, w, b)
    got = ci8.layer_norm_backward(dy, x, w, mean, rstd)
    bounds = ref.layer_norm_backward(dy, x, w, mean, rstd)
    for i, base in enumerate((x, w, b)):
        v = torch.randn(*base.shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(s):
            p = [t.double() for t in (x, w, b)]
            p[i] = p[i] + s * v
            return (dy.double() * ref.layer_norm(p[0], p[1], p[2])["y"][0]).sum()

        diff = float((loss(h) - loss(-h)) / (2 * h))
        mine = float((got[i].double() * v).sum())
        # mean and rstd are 32-bit: another 2^-20 of the magnitudes
        tol = float(((bounds[i][1] + 2.0 ** -20 * got[i].double().abs()) * v.abs()).sum()) + 100 * h * h * m * d
        assert abs(diff - mine) <= tol, (i, diff, mine, tol)


def test_sums_do_not_depend_on_the_run(ci8):
    """The same call twice gives the same bits (no atomics)."""
    g = gen(15)
    x, w, dy, z = values(g, 700, 264), values(g, 520, 264), values(g, 700, 520), values(g, 700, 520)
    a, b = (ci8.linear_backward(dy, x, w, preact=z, activation="gelu") for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    y, mean, rstd = ci8.layer_norm(x)
    a, b = (ci8.layer_norm_backward(x, x, None, mean, rstd) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_other_stream(ci8):
    """Operators on a stream of their own, given as `stream` or made current."""
    g = gen(16)
    x, w = values(g, 300, 259), values(g, 200, 259)
    want = ci8.linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = ci8.linear(x, w, stream=s)
    n = ci8.layer_norm(x, stream=s)
    with torch.cuda.stream(s):
        z = ci8.linear(x, w)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want)
    assert torch.equal(n[0], ci8.layer_norm(x)[0])


def test_graph_replays(ci8):
    """One feed-forward block, forward and backward, recorded into a graph and
    replayed on changing inputs, with eager work between the replays."""
    g = gen(17)
    m, d, n = 96, 136, 264
    x, w1, w2, dy = values(g, m, d), values(g, n, d, scale=0.1), values(g, d, n, scale=0.1), values(g, m, d)
    gamma, b1 = values(g, d), values(g, n)

    def block():
        h, mean, rstd = ci8.layer_norm(x, gamma)
        z = torch.empty(m, n, dtype=BF16, device="cuda")
        a = ci8.linear(h, w1, b1, activation="gelu_tanh", preact=z)
        y = ci8.linear(a, w2, residual=x)
        da, dw2, _ = ci8.linear_backward(dy, a, w2, need_dbias=False)
        dh, dw1, db1 = ci8.linear_backward(da, h, w1, preact=z, activation="gelu_tanh")
        dx, dg, _ = ci8.layer_norm_backward(dh, x, gamma, mean, rstd)
        return y, dw2, dw1, db1, dx, dg

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            block()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block()
    for i in range(4):
        x.copy_(values(gen(100 + i), m, d))
        dy.copy_(values(gen(200 + i), m, d))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, block()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_offsets_past_32_bits(ci8):
    """Outputs, rows and gradients beyond 2^31 elements: spot rows against the
    64-bit form."""
    m, n, k = 70000, 32768, 64
    g = gen(18)
    x, w, b = values(g, m, k), values(g, n, k, scale=0.1), values(g, n)
    print(f"[gpu] linear {m}x{n}x{k}", flush=True)
    y = ci8.linear(x, w, b, activation="silu")
    rows = [0, 1, 255, 65535, 65536, 69999]
    (v, e), _ = ref.linear(x[rows], w, b, "silu", out_dtype=BF16)
    ref.check(y[rows], v, e, "linear rows")
    print(f"[gpu] layer_norm {m}x{n}", flush=True)
    h, mean, rstd = ci8.layer_norm(y)
    want = ref.layer_norm(y[rows])
    ref.check(h[rows], want["y"][0], want["y"][1] + ref.rounding(want["y"][0].abs() + want["y"][1], BF16), "norm rows")
    print(f"[gpu] linear_backward {m}x{n}x{k}", flush=True)
    dx, dw, db = ci8.linear_backward(h, x, w)
    (v, e), _, _ = ref.linear_backward(h[rows], x[rows], w)
    ref.check(dx[rows], v, e, "dx rows")
    cols = [0, 1, 511, 32767]
    _, (v, e), (bv, be) = ref.linear_backward(h[:, cols].contiguous(), x, w[cols])
    ref.check(dw[cols], v, e, "dw rows")
    ref.check(db[cols], bv, be, "dbias")
    print(f"[gpu] layer_norm_backward {m}x{n}", flush=True)
    dxn, _, _ = ci8.layer_norm_backward(h, y, None, mean, rstd)
    (v, e), _, _ = ref.layer_norm_backward(h[rows], y[rows], None, mean[rows], rstd[rows])
    ref.check(dxn[rows], v, e, "norm dx rows")


@pytest.mark.parametrize("dtype", [BF16, FP16, I8])
@pytest.mark.parametrize("tile", ["128x128d", "128x128d/2", "128x128d/3"])
@pytest.mark.parametrize("m,n,k", [(128, 128, 64), (300, 200, 160), (65, 513, 1056), (257, 264, 4096), (130, 100, 24)])
def test_linear_deep_ring(ci8, monkeypatch, dtype, tile, m, n, k):
    """The five-slot ring with fewer, as many and more stages than slots."""
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    run_linear(ci8, m, n, k, dtype, act=ACTS[(m + k // 32) % 5], residual=m % 2 == 0, keep=True)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("m,n,k", [(520, 264, 300), (289, 1040, 96)])
def test_backward_deep_ring(ci8, monkeypatch, dtype, m, n, k):
    monkeypatch.setenv("CONV_I8_DENSE_TILE", "128x128d")
    run_backward(ci8, m, n, k, dtype, "silu")


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("m,n,k", [(777, 520, 264), (64, 64, 64), (130, 9, 1000), (7, 1000, 130), (2, 3, 5)])
def test_backward_pair(ci8, m, n, k, act):
    """Both products and the bias gradient in one launch, and the same bits when each is asked for alone."""
    from int8_convolution_forward_amd.dense import linear_backward_plan
    run_backward(ci8, m, n, k, BF16, act)
    g = gen(21)
    dy, x, w, z = values(g, m, n), values(g, m, k), values(g, n, k), values(g, m, n)
    plan = linear_backward_plan(dy, x, w, preact=z, activation=act)
    assert "launches=paired" in plan, plan
    assert "launches=apart" in linear_backward_plan(dy, x, w, preact=z, activation=act, need_dx=False)
    full = ci8.linear_backward(dy, x, w, preact=z, activation=act)
    for i in range(3):
        part = ci8.linear_backward(dy, x, w, preact=z, activation=act, need_dx=i == 0, need_dw=i == 1, need_dbias=i == 2)
        assert torch.equal(part[i], full[i])


# more rows than thread groups, so that each walks over several
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("m,d", [(2500, 4096), (2300, 4001), (1500, 9001), (1200, 16384), (4500, 777), (9000, 130), (9001, 8),
                                 (5000, 11), (3000, 6), (1030, 20000)])
def test_norm_many_rows(ci8, dtype, m, d):
    run_norm(ci8, m, d, dtype, weight=d % 3 != 0)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("m,d", [(1100, 4096), (1100, 4001), (1050, 8192), (1041, 8191), (1030, 12345), (9000, 130), (3000, 7),
                                 (600, 9), (5000, 8)])
def test_norm_backward_many_rows(ci8, dtype, m, d):
    run_norm_backward(ci8, m, d, dtype, weight=d % 3 != 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n", [(1, 513), (37, 520), (70, 1001), (130, 7), (66, 8), (19, 1024)])
def test_backward_bias_only(ci8, m, n, act):
    """The pass over dy and z at whole, partial and narrow strips of columns."""
    run_backward(ci8, m, n, 8, BF16, act, dy_layout=dict(pitch=n % 3), z_layout=dict(pitch=5))
    g = gen(22)
    dy, z = values(g, m, n, dtype=FP16), values(g, m, n, dtype=FP16, scale=2.0)
    x, w = values(g, m, 8, dtype=FP16), values(g, n, 8, dtype=FP16)
    got = ci8.linear_backward(dy, x, w, preact=z, activation=act, need_dx=False, need_dw=False)[2]
    ref.check(got, *ref.linear_backward(dy, x, w, z if act != "none" else None, act)[2], "dbias")


def test_gelu_tanh_far_values(ci8):
    """Pre-activations up to the type's largest: no overflow inside the gate, its slope or their products."""
    big = torch.tensor([0.0, 5, -5, 12, -12, 100, -100, 1e4, -1e4, 1e15, -1e15, 1e19, -1e19, 3e38, -3e38], device="cuda").to(BF16)
    n = big.numel()
    one = torch.ones(40, 1, dtype=BF16, device="cuda")
    for m in (2, 40):
        y = ci8.linear(one[:m], big[:, None].contiguous(), activation="gelu_tanh")
        want = ref.act(big.double(), "gelu_tanh")
        assert bool(torch.isfinite(y).all())
        ref.check(y, want.expand(m, n), (ref.ACT_ERR * big.double().abs() + ref.rounding(want.abs(), BF16)).expand(m, n), "far")
    z = big.expand(4, n).contiguous()
    db = ci8.linear_backward(torch.ones_like(z), one[:4], big[:, None].contiguous(), preact=z, activation="gelu_tanh",
                             need_dx=False, need_dw=False)[2]
    far = big.double().abs() >= 100
    assert torch.equal(db[far].double(), 4.0 * (big[far] > 0).double())
