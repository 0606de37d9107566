"""Layer norm at the ends of the number range."""
import pytest
import torch

from tests import dense_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
WIDTHS = (1, 7, 9, 12, 100, 256, 600, 1100, 2048, 2100, 5000, 9004, 17000)


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("m", [3, 1500])
def test_mean_times_rstd_past_the_largest_number(ci8, d, m):
    """Constant rows of 2^113, whose sums are exact, with rstd = 10^6: every xh is 0, and what a thread holds past
    the row's end must not become 0 times infinity."""
    x = torch.full((m, d), 2.0 ** 113, dtype=FP32, device="cuda")
    b = torch.arange(d, dtype=FP32, device="cuda") % 5 - 2
    y, mean, rstd = ci8.layer_norm(x, None, b, eps=1e-12)
    assert bool((mean == 2.0 ** 113).all()) and bool((rstd > 9e5).all())
    assert torch.equal(y, b.expand(m, d))
    q, s = ci8.layer_norm_i8(x, None, b, eps=1e-12)
    ref.check(s, (b.abs().max().double() / 127).expand(m), torch.full((m,), 2.0 ** -24, dtype=torch.float64, device="cuda"),
              "scale")
    assert torch.equal(q, (b * 127 / b.abs().max()).round().to(torch.int8).expand(m, d))
    dy = torch.randn(m, d, generator=torch.Generator(device="cuda").manual_seed(111), device="cuda")
    got = ci8.layer_norm_backward(dy, x, None, mean, rstd)
    for name, t, (v, e) in zip(("dx", "dweight", "dbias"), got, ref.layer_norm_backward(dy, x, None, mean, rstd)):
        if name != "dx":  # the bound of dx has xh's rounding, 2^113 times what it is here
            ref.check(t, v, e, name)
    c = dy.double()
    v = rstd.double()[:, None] * (c - c.mean(1, keepdim=True))
    e = rstd.double()[:, None] * (ref._steps(d) + 6) * ref.F32 * (c.abs() + c.abs().mean(1, keepdim=True))
    ref.check(got[0], v, e, "dx")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [7, 12, 600, 4096, 9004, 66000])
@pytest.mark.parametrize("size", [2.0 ** -99, 2.0 ** -101, 2.0 ** -118, 2.0 ** -122, 2.0 ** -126])
def test_int8_rows_of_tiny_values(ci8, dtype, d, size):
    """Weights near the smallest normal number: the row still takes all of 8 bits, and q * scale gives it back.
    Below the normal range numbers have steps of 2^-149, of which half may be lost in y and in 127 scales."""
    g = torch.Generator(device="cuda").manual_seed(112)
    x = torch.randn(5, d, generator=g, device="cuda").to(dtype)
    w = torch.full((d,), size, dtype=dtype, device="cuda")
    q, s = ci8.layer_norm_i8(x, w)
    want = ref.layer_norm(x, w)
    v, e = want["y"]
    top = v.abs().amax(1)
    es = e.amax(1) / 127 + 2 * ref.F32 * (top / 127) + 2.0 ** -149
    ref.check(s, top / 127, es, "scale")
    assert bool((q.abs().amax(1) == 127).all())
    exact = v * 127 / top[:, None]  # what is rounded, off by its own error and that of the largest value
    off = 127 * (e + 2.0 ** -149) / top[:, None] * 2 + 2 ** -10
    ref.check(q.double(), exact, 0.5 + off, "q")
    ref.check(q.double() * s.double()[:, None], v, (0.5 + off) * (top / 127)[:, None] + 127 * es[:, None], "q * scale")
