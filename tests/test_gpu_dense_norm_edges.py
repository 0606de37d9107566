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
