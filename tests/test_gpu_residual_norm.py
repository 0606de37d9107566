"""The norm fused with a residual connection and its gradients on the GPU,
against 64 bits."""
import math

import pytest
import torch

from tests import block_reference as ref
from tests.dense_reference import check, rounding

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def say(*a):
    print("[gpu]", *a, flush=True)


def inputs(m, d, dtype, gates, post, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * m + d + seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (n(m, d) * 1.5 + n(m, 1) * 2).to(dtype)
    h = (n(m, d) * 0.5 + n(m, 1)).to(dtype)
    gate = None if gates is None else n(d).to(dtype) if gates == 0 else n(gates, d).to(dtype)
    return dict(x=x, h=h, weight=(1 + 0.2 * n(d)).to(dtype), bias=n(d).to(dtype), gate=gate,
                post_weight=(1 + 0.2 * n(d)).to(dtype) if post else None, dr=n(m, d).to(dtype), dy=n(m, d).to(dtype))


def check_forward(ci8, t, scale, kind, label, eps=1e-5, given=()):
    """r against the formula; y and the statistics against the norm of the r that came back."""
    args = {k: t[k] for k in ("weight", "bias", "gate", "post_weight")}
    r, y, stats = ci8.residual_norm(t["x"], t["h"], **args, scale=scale, norm=kind, eps=eps)
    m, dt = t["x"].shape[0], t["x"].dtype
    v, e = ref.residual(t["x"], t["h"], t["gate"], t["post_weight"], scale, kind, eps)
    check(r, v, e + rounding(v.abs() + e, dt), (*label, "r"))
    n = ref.norm(r, t["weight"], t["bias"], kind, eps)
    check(y, n["y"][0], n["y"][1] + rounding(n["y"][0].abs() + n["y"][1], dt), (*label, "y"))
    check(stats[0], *n["mean"], (*label, "mean"))
    check(stats[1], *n["rstd"], (*label, "rstd"))
    assert stats.shape == (4 if t["post_weight"] is not None else 2, m)
    if t["post_weight"] is not None:
        n = ref.norm(t["h"], None, None, kind, eps)
        check(stats[2], *n["mean"], (*label, "post mean"))
        check(stats[3], *n["rstd"], (*label, "post rstd"))
    r8, q, s = ci8.residual_norm_fp8(t["x"], t["h"], **args, scale=scale, norm=kind, eps=eps)
    assert torch.equal(r8, r)
    n = ref.norm(r, t["weight"], t["bias"], kind, eps)["y"]
    v, e = ref.quantized_within(n[0], n[1], torch.float8_e4m3fn)
    check(ref.values(q, s), v, e, (*label, "q"))
    return r, y, stats


def check_backward(ci8, t, r, stats, scale, kind, label):
    got = ci8.residual_norm_backward(t["dr"], t["dy"], r, t["h"], stats, weight=t["weight"], gate=t["gate"],
                                     post_weight=t["post_weight"], scale=scale, norm=kind)
    want = ref.residual_backward(t["dr"], t["dy"], r, t["h"], stats, t["weight"], t["gate"], t["post_weight"], scale, kind)
    for name, g in zip(("dx", "dh", "dweight", "dbias", "dgate", "dpost_weight"), got):
        assert (g is None) == (name not in want), (*label, name)
        if g is not None:
            check(g, *want[name], (*label, name))
    return got


SIZES = [(1, 1), (3, 7), (5, 8), (1, 64), (4, 127), (12, 128), (30, 511), (33, 512), (8, 513), (1500, 520), (6, 1024), (1100, 1000),
         (9, 1537), (7, 2048), (600, 2056), (10, 4096), (4, 4097), (3, 8192), (5, 8193), (2, 16384), (3, 16385), (2, 33000)]


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_sizes(ci8, m, d, dtype):
    for kind, gates, post in (("layer", 0, True), ("rms", None, False), ("rms", m, True), ("layer", 1, False)):
        t = inputs(m, d, DTYPES[dtype], gates, post)
        label = (m, d, dtype, kind, gates, post)
        say("residual_norm", *label)
        r, _, stats = check_forward(ci8, t, 0.75, kind, label)
        check_backward(ci8, t, r, stats, 0.75, kind, label)


@pytest.mark.parametrize("gates", [1, 2, 3, 6, 30, 300, 600])
@pytest.mark.parametrize("d", [96, 700, 1544, 2600, 5000, 9000])
def test_gates_of_groups_of_rows(ci8, gates, d):
    """Few groups share workgroups' partial sums, many are summed by a workgroup each."""
    for post in (False, True):
        t = inputs(600, d, torch.bfloat16, gates, post, seed=gates)
        label = (gates, d, post)
        say("residual_norm", *label)
        r, _, stats = check_forward(ci8, t, 1.0, "layer", label)
        check_backward(ci8, t, r, stats, 1.0, "layer", label)


def test_many_rows(ci8):
    for m, d in ((20000, 64), (5000, 1024), (3000, 2048), (2500, 4096)):
        t = inputs(m, d, torch.bfloat16, 4, True)
        r, _, stats = check_forward(ci8, t, 1.0, "rms", (m, d))
        check_backward(ci8, t, r, stats, 1.0, "rms", (m, d))


@pytest.mark.parametrize("d", [5, 64, 1000, 3000, 6000, 9000])
def test_without_a_block_before(ci8, d):
    """h None: a norm alone; dr None; no weights."""
    for kind in ("layer", "rms"):
        t = inputs(37, d, torch.float16, None, False)
        r, y, stats = ci8.residual_norm(t["x"], None, t["weight"], t["bias"], norm=kind)
        assert r is t["x"] or r.data_ptr() == t["x"].data_ptr()
        n = ref.norm(r, t["weight"], t["bias"], kind)
        check(y, n["y"][0], n["y"][1] + rounding(n["y"][0].abs() + n["y"][1], y.dtype), (d, kind))
        t.update(h=None, dr=None)
        check_backward(ci8, t, r, stats, 1.0, kind, (d, kind))
        t.update(weight=None)
        _, y, stats = ci8.residual_norm(t["x"], None, norm=kind)
        n = ref.norm(r, None, None, kind)
        check(y, n["y"][0], n["y"][1] + rounding(n["y"][0].abs() + n["y"][1], y.dtype), (d, kind))
        check_backward(ci8, t, r, stats, 1.0, kind, (d, kind))


def test_parts_of_the_gradients(ci8):
    t = inputs(50, 300, torch.bfloat16, 5, True)
    r, _, stats = check_forward(ci8, t, 2.0, "layer", ())
    full = check_backward(ci8, t, r, stats, 2.0, "layer", ())
    kw = dict(weight=t["weight"], gate=t["gate"], post_weight=t["post_weight"], scale=2.0)
    part = ci8.residual_norm_backward(t["dr"], t["dy"], r, t["h"], stats, need_params=False, **kw)
    assert torch.equal(part[0], full[0]) and torch.equal(part[1], full[1]) and part[2:] == (None,) * 4
    zero = ci8.residual_norm_backward(torch.zeros_like(t["dr"]), t["dy"], r, t["h"], stats, **kw)
    none = ci8.residual_norm_backward(None, t["dy"], r, t["h"], stats, **kw)
    assert all(torch.equal(a, b) for a, b in zip(zero, none))


def test_layouts(ci8):
    t = inputs(24, 200, torch.bfloat16, None, True)
    kw = dict(weight=t["weight"], bias=t["bias"], post_weight=t["post_weight"], scale=0.5)
    g = torch.Generator(device="cuda").manual_seed(8)
    gate = torch.randn(4, 200, generator=g, device="cuda").to(torch.bfloat16)
    r, y, stats = ci8.residual_norm(t["x"], t["h"], gate=gate, **kw)
    batch = lambda v: v.reshape(4, 6, 200)  # noqa: E731
    rb, yb, sb = ci8.residual_norm(batch(t["x"]), batch(t["h"]), gate=gate.reshape(2, 2, 200), **kw)
    assert torch.equal(rb.reshape(24, 200), r) and torch.equal(yb.reshape(24, 200), y) and sb.shape == (4, 4, 6)
    assert torch.equal(sb.reshape(4, 24), stats)
    far = torch.zeros(24, 333, dtype=torch.bfloat16, device="cuda")
    far[:, 7:207] = t["x"]
    for x, h, w in ((far[:, 7:207], t["h"], t["weight"]), (t["x"].t().contiguous().t(), t["h"], t["weight"]),
                    (t["x"], t["h"].t().contiguous().t(), torch.stack([t["weight"]] * 3, 1)[:, 1])):
        a = ci8.residual_norm(x, h, gate=gate, **{**kw, "weight": w})
        assert all(torch.equal(p, q) for p, q in zip(a, (r, y, stats)))
    dr, dy = t["dr"], t["dy"]
    full = ci8.residual_norm_backward(dr, dy, r, t["h"], stats, gate=gate, weight=t["weight"],
                                      post_weight=t["post_weight"], scale=0.5)
    part = ci8.residual_norm_backward(batch(dr), batch(dy), batch(r), batch(t["h"]), sb, gate=gate.reshape(2, 2, 200),
                                      weight=t["weight"], post_weight=t["post_weight"], scale=0.5)
    for a, b in zip(part, full):
        assert torch.equal(a.reshape(b.shape), b)
    assert part[4].shape == (2, 2, 200)
    # a gradient expanded from one row, statistics with a stride
    one = dy[:1].expand(24, 200)
    a = ci8.residual_norm_backward(one, one, r, t["h"], torch.stack([stats] * 2, 2)[..., 0], gate=gate, weight=t["weight"],
                                   post_weight=t["post_weight"], scale=0.5)
    b = ci8.residual_norm_backward(one.contiguous(), one.contiguous(), r, t["h"], stats, gate=gate, weight=t["weight"],
                                   post_weight=t["post_weight"], scale=0.5)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    empty = ci8.residual_norm(t["x"][:0], t["h"][:0], **kw)
    assert empty[0].shape == (0, 200) and empty[2].shape == (4, 0)
    back = ci8.residual_norm_backward(dr[:0], dy[:0], r[:0], t["h"][:0], stats[:, :0], gate=gate, weight=t["weight"],
                                      post_weight=t["post_weight"])
    assert back[0].shape == (0, 200) and not any(bool(v.any()) for v in back[2:]) and back[4].shape == (4, 200)


def test_refusals(ci8):
    t = inputs(24, 200, torch.bfloat16, 5, False)
    with pytest.raises(ci8.ConvI8Error) as e:
        ci8.residual_norm(t["x"], t["h"], gate=t["gate"])  # five rows do not divide 24
    assert e.value.name == "CONV_I8_ERR_DIMS"
    with pytest.raises(ci8.ConvI8Error):
        ci8.residual_norm(t["x"], t["h"].reshape(12, 400))
    with pytest.raises(ci8.ConvI8Error):
        ci8.residual_norm(t["x"], t["h"].float())
    with pytest.raises(ci8.ConvI8Error):
        ci8.residual_norm(t["x"], None, gate=t["gate"][0])
    with pytest.raises(ci8.ConvI8Error):
        ci8.residual_norm_backward(t["dr"], t["dy"], t["x"], t["h"], torch.zeros(3, 23, device="cuda"))


def test_edges_of_the_range(ci8):
    """A constant row, one far from zero, infinities and NaN: they stay in their row."""
    for d in (40, 1000, 5000, 9000):
        for kind in ("layer", "rms"):
            t = inputs(8, d, torch.float32, None, True)
            t["x"][0], t["h"][0] = 3.0, 0.0
            t["x"][1] += 4096.0
            t["h"][2, 1] = math.inf
            t["x"][3, d - 1] = math.nan
            t["h"][4] = 7.0
            r, y, stats = ci8.residual_norm(t["x"], t["h"], t["weight"], t["bias"], post_weight=t["post_weight"], norm=kind)
            _, q, s = ci8.residual_norm_fp8(t["x"], t["h"], t["weight"], t["bias"], post_weight=t["post_weight"], norm=kind)
            fine = [0, 1, 4, 5, 6, 7]
            keep = {k: v[fine] if k in ("x", "h", "dr", "dy") else v for k, v in t.items()}
            a = ci8.residual_norm(keep["x"], keep["h"], t["weight"], t["bias"], post_weight=t["post_weight"], norm=kind)
            assert torch.equal(a[0], r[fine]) and torch.equal(a[1], y[fine]) and torch.equal(a[2], stats[:, fine])
            assert bool(torch.isfinite(y[fine]).all()) and bool(torch.isnan(y[2]).any()) and bool(torch.isnan(y[3]).all())
            assert bool(torch.isfinite(ref.values(q, s)[fine]).all()) and bool(torch.isnan(ref.values(q, s)[3]).all())
            check_forward(ci8, keep, 1.0, kind, (d, kind))


@pytest.mark.parametrize("d", [5, 40, 1000, 2048, 5000, 9000, 17000])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_whose_squares_32_bits_do_not_hold(ci8, d, kind, dtype):
    """They are NaN, by either norm and in the gradients, and stay in their row; right up to there."""
    t = inputs(8, d, DTYPES[dtype], None, True)
    usual = ci8.residual_norm(t["x"], t["h"], t["weight"], t["bias"], post_weight=t["post_weight"], norm=kind)
    for name, row in (("x", 2), ("h", 5)):
        for big in (1e25, 3e30):
            v = {**t, name: t[name].clone()}
            v[name][row] = (v[name][row].float() * big).to(DTYPES[dtype])
            args = (v["x"], v["h"], t["weight"], t["bias"])
            say("residual_norm", d, kind, dtype, name, big)
            r, y, stats = ci8.residual_norm(*args, post_weight=t["post_weight"], norm=kind)
            _, q, s = ci8.residual_norm_fp8(*args, post_weight=t["post_weight"], norm=kind)
            others = [i for i in range(8) if i != row]
            assert bool(torch.isnan(y[row]).all()) and bool(torch.isnan(stats[1, row]))
            assert bool(torch.isnan(ref.values(q, s)[row]).all())
            assert bool(torch.isfinite(r[row]).all()) == (name == "x") and bool(torch.isnan(stats[3, row])) == (name == "h")
            assert all(torch.equal(a[..., others] if a is stats else a[others], b[..., others] if a is stats else b[others])
                       for a, b in zip((r, y, stats), usual))
            dx, dh, *_ = ci8.residual_norm_backward(t["dr"], t["dy"], r, v["h"], stats, t["weight"], post_weight=t["post_weight"],
                                                    norm=kind)
            assert bool(torch.isnan(dx[row]).all()) and bool(torch.isfinite(dx[others]).all()) and bool(torch.isfinite(dh[others]).all())
    # 2^60 / sqrt(d), with the values of `inputs` up to 2^4 of it
    fits = inputs(8, d, DTYPES[dtype], None, True)
    up = 2.0 ** math.floor(60 - 0.5 * math.log2(d))
    fits["x"], fits["h"] = (fits["x"] * up), (fits["h"] * up)
    check_forward(ci8, fits, 0.75, kind, (d, dtype, kind))


@pytest.mark.parametrize("d", [70, 1100, 9000])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradients_against_differences(ci8, d, kind):
    """sum(dr r + dy y), 64-bit differences of the formula along random directions against the gradients in 32 bits.
    Along a direction the central difference is off by step^2 / 6 of the third derivative (1e-8 here), the
    gradients' sum by the bounds of its terms."""
    t = inputs(12, d, torch.float32, 3, True)
    r, _, stats = ci8.residual_norm(t["x"], t["h"], t["weight"], t["bias"], t["gate"], t["post_weight"], scale=0.7, norm=kind)
    got = ci8.residual_norm_backward(t["dr"], t["dy"], r, t["h"], stats, t["weight"], t["gate"], t["post_weight"], 0.7, kind)
    names = ("x", "h", "weight", "bias", "gate", "post_weight")
    grads = dict(zip(("x", "h", "weight", "bias", "gate", "post_weight"), got))
    base = {k: t[k].double() for k in names}

    def normed(v):
        mean = v.mean(1, keepdim=True) if kind == "layer" else 0
        return (v - mean) / torch.sqrt((v - mean).square().mean(1, keepdim=True) + 1e-5)

    def loss(p):
        s = float(torch.tensor(0.7)) * p["x"] + p["gate"].repeat_interleave(4, 0) * normed(p["h"]) * p["post_weight"]
        return (t["dr"].double() * s + t["dy"].double() * (normed(s) * p["weight"] + p["bias"])).sum()

    g = torch.Generator(device="cuda").manual_seed(77)
    for name in names:
        v = torch.randn(base[name].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-4
        diff = (loss({**base, name: base[name] + step * v}) - loss({**base, name: base[name] - step * v})) / (2 * step)
        along = (grads[name].double() * v).sum()
        size = (grads[name].double() * v).abs().sum()
        assert abs(float(diff - along)) <= 1e-5 * float(size), (name, float(diff), float(along), float(size))


def test_same_bits_again(ci8):
    t = inputs(2000, 1024, torch.bfloat16, 4, True)
    a = ci8.residual_norm(t["x"], t["h"], t["weight"], t["bias"], t["gate"], t["post_weight"])
    b = ci8.residual_norm_backward(t["dr"], t["dy"], a[0], t["h"], a[2], t["weight"], t["gate"], t["post_weight"])
    for _ in range(3):
        c = ci8.residual_norm(t["x"], t["h"], t["weight"], t["bias"], t["gate"], t["post_weight"])
        assert all(torch.equal(p, q) for p, q in zip(a, c))
        c = ci8.residual_norm_backward(t["dr"], t["dy"], a[0], t["h"], a[2], t["weight"], t["gate"], t["post_weight"])
        assert all(torch.equal(p, q) for p, q in zip(b, c))


def test_many_long_rows(ci8):
    """More rows, of more columns than the registers hold, than there are workgroups: each takes several
    one after the other.  The rows overlap in memory, so that windows of one sum of squares give their norms."""
    m, d = 65536 + 512, 16392
    say("many long rows", m, d)
    g = torch.Generator(device="cuda").manual_seed(5)
    values = torch.randn(8 * m + d, generator=g, device="cuda")
    values *= torch.exp2(torch.linspace(-20, 20, values.numel(), device="cuda"))
    values = values.to(torch.bfloat16)
    x = values.as_strided((m, d), (8, 1))
    r, y, stats = ci8.residual_norm(x, None, eps=0.0, norm="rms")
    total = torch.cat([torch.zeros(1, device="cuda", dtype=torch.float64), values.double().square().cumsum(0)])
    at = torch.arange(m, device="cuda") * 8
    rstd = ((total[at + d] - total[at]) / d).rsqrt()
    # d + 1 roundings of a sum of positive terms in 32 bits, halved by the root, and three of the quotient and the root
    assert bool(((stats[1].double() / rstd - 1).abs() <= (d / 2 + 4) * 2.0 ** -24).all())
    for row in (0, 1, 65535, 65536, m - 1):
        want = x[row].double() * rstd[row]
        bound = want.abs() * (2.0 ** -8 + (d / 2 + 8) * 2.0 ** -24)
        assert bool(((y[row].double() - want).abs() <= bound).all())
