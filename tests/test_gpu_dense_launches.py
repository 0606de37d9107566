"""Sizes whose plain launches would pass 2^32 threads, and rows of one to seven
columns, which have kernels of their own."""
import pytest
import torch

from tests import dense_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def rows(g, m, d, dtype, pitch=0):
    """[m, d] in a buffer whose gaps hold NaN."""
    buf = torch.full((m, d + pitch), float("nan"), dtype=dtype, device="cuda")
    buf[:, :d] = torch.randn(m, d, generator=g, device="cuda") * 1.5 + 1
    return buf[:, :d]


def check_norm(ci8, m, d, dtype, pitch=0, params=True):
    print(f"[gpu] layer norm and gradients m={m} d={d} {dtype} pitch={pitch} params={params}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(51)
    x, dy = rows(g, m, d, dtype, pitch), rows(g, m, d, dtype, pitch)
    w, b = (torch.randn(2, d, generator=g, device="cuda").to(dtype)) if params else (None, None)
    want = ref.layer_norm(x, w, b)
    v, e = want["y"]
    y, mean, rstd = ci8.layer_norm(x, w, b)
    q, s = ci8.layer_norm_i8(x, w, b)
    got = ci8.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    ref.check(mean, *want["mean"], "mean")
    ref.check(rstd, *want["rstd"], "rstd")
    ref.check(y, v, e + ref.rounding(v.abs() + e, dtype), "y")
    top, es = v.abs().amax(1), e.amax(1) / 127 + 2 * ref.F32 * (v.abs().amax(1) / 127)
    ref.check(s, top / 127, es, "scale")
    ref.check(q.double() * s.double()[:, None], v, 0.5 * (top / 127 + es)[:, None] * (1 + 2 ** -10) + e + 127 * es[:, None],
              "q * scale")
    for name, t, (gv, gb) in zip(("dx", "dweight", "dbias"), got, ref.layer_norm_backward(dy, x, w, mean, rstd)):
        ref.check(t, gv, gb, name)
    alone = ci8.layer_norm_backward(dy, x, w, mean, rstd, need_params=False)
    assert torch.equal(alone[0], got[0]) and alone[1] is None and alone[2] is None


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("d", [1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("m", [1, 63, 257, 1025, 200003])
def test_narrow_rows(ci8, dtype, d, m):
    check_norm(ci8, m, d, dtype, pitch=m % 3, params=d != 4)


@pytest.mark.parametrize("d", [3, 7])
def test_four_million_narrow_rows(ci8, d):
    check_norm(ci8, (1 << 22) + 3, d, BF16)


def test_many_rows_of_eight_columns(ci8):
    """2^21 workgroups of four rows at a time, each of which walks over several."""
    check_norm(ci8, (1 << 24) + 5, 8, BF16)


@pytest.mark.parametrize("d", [16385, 65537])
def test_many_wide_rows(ci8, d):
    """More rows than the 2^16 workgroups of 1024 threads: spot rows, among them those taken second."""
    m = (1 << 16) + 3
    print(f"[gpu] layer norm and gradients m={m} d={d}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(55)
    x, dy = (torch.randn(m, d, generator=g, device="cuda", dtype=BF16) for _ in range(2))
    at = [0, 1, 2, 65535, 65536, 65537, 65538]
    want = ref.layer_norm(x[at])
    v, e = want["y"]
    y, mean, rstd = ci8.layer_norm(x)
    ref.check(y[at], v, e + ref.rounding(v.abs() + e, BF16), "y")
    del y
    q, s = ci8.layer_norm_i8(x)
    top, es = v.abs().amax(1), e.amax(1) / 127 + 2 * ref.F32 * (v.abs().amax(1) / 127)
    ref.check(s[at], top / 127, es, "scale")
    ref.check(q[at].double() * s[at].double()[:, None], v,
              0.5 * (top / 127 + es)[:, None] * (1 + 2 ** -10) + e + 127 * es[:, None], "q * scale")
    del q
    dx, _, _ = ci8.layer_norm_backward(dy, x, None, mean, rstd, need_params=False)
    (v, e), _, _ = ref.layer_norm_backward(dy[at], x[at], None, mean[at], rstd[at])
    ref.check(dx[at], v, e, "dx")


def test_bias_gradient_of_very_many_columns(ci8):
    """2^27 columns are 2^32 threads of the columns' sums."""
    n = (1 << 27) + 40
    print(f"[gpu] bias gradient of {n} columns", flush=True)
    g = torch.Generator(device="cuda").manual_seed(52)
    dy = torch.randn(2, n, generator=g, device="cuda", dtype=BF16)
    x, w = torch.zeros(2, 1, dtype=BF16, device="cuda"), torch.zeros(n, 1, dtype=BF16, device="cuda")
    _, _, db = ci8.linear_backward(dy, x, w, need_dx=False, need_dw=False)
    assert torch.equal(db, (dy[0].float() + dy[1].float()).to(BF16))


def test_one_token_to_very_many_columns(ci8):
    n = (1 << 26) + 24
    print(f"[gpu] linear 1 x {n}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(53)
    x, w = torch.randn(1, 8, generator=g, device="cuda").to(BF16), torch.randn(n, 8, generator=g, device="cuda").to(BF16)
    y = ci8.linear(x, w)
    # eight products of 16-bit values in 32 bits: the bound of the 64-bit form, column by column
    v = (w.double() * x.double()).sum(1)
    e = 9 * ref.F32 * (w.double() * x.double()).abs().sum(1)
    ref.check(y[0], v, e + ref.rounding(v.abs() + e, BF16), "y")


def test_norm_gradients_of_a_very_wide_row(ci8):
    """2 (2^26 + 8) columns of partial sums are more than 2^32 threads."""
    d = (1 << 26) + 8
    print(f"[gpu] layer norm gradients d={d}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(54)
    x, dy = (torch.randn(2, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    mean, rstd = torch.tensor([0.25, -0.5], device="cuda"), torch.tensor([0.75, 1.5], device="cuda")
    dx, dw, db = ci8.layer_norm_backward(dy, x, None, mean, rstd)
    for name, t, (v, b) in zip(("dx", "dweight", "dbias"), (dx, dw, db), ref.layer_norm_backward(dy, x, None, mean, rstd)):
        ref.check(t, v, b, name)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("m,d", [(1024, 64), (1024, 1000), (1023, 777), (1025, 777), (1000, 2048), (1024, 8192), (513, 8192),
                                 (512, 8200), (513, 8200), (512, 16384), (511, 9001)])
def test_gradients_on_both_sides_of_one_launch(ci8, dtype, m, d):
    check_norm(ci8, m, d, dtype, pitch=m % 2)
