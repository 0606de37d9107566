"""The dense entries on a stream that is not the operands' own."""
from types import SimpleNamespace

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def calls(ci8, m, stream):
    """Operands by name, and the call on them, of every entry."""
    g = torch.Generator(device="cuda").manual_seed(91)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    i8 = lambda *s: torch.randint(-9, 9, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)  # noqa: E731
    f = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    return [
        (lambda t: ci8.linear(t[0], t[1], t[2], residual=t[3], stream=stream), [r(m, 512), r(256, 512), r(256), r(m, 256)]),
        (lambda t: ci8.linear(t[0], t[1], x_scale=t[2], w_scale=t[3], stream=stream), [i8(m, 512), i8(256, 512), f(m), f(256)]),
        (lambda t: ci8.linear_backward(t[0], t[1], t[2], preact=t[3], activation="silu", stream=stream),
         [r(m, 256), r(m, 512), r(256, 512), r(m, 256)]),
        (lambda t: ci8.layer_norm(t[0], t[1], t[2], stream=stream), [r(m, 512), r(512), r(512)]),
        (lambda t: ci8.layer_norm_i8(t[0], t[1], t[2], stream=stream), [r(m, 512), r(512), r(512)]),
        (lambda t: ci8.layer_norm_backward(t[0], t[1], t[2], t[3], t[4], stream=stream),
         [r(m, 512), r(m, 512), r(512), f(m), f(m)]),
    ]


@pytest.mark.parametrize("m", [5, 700])
def test_operands_freed_before_the_stream_has_read_them(ci8, m):
    """Their memory is not handed to other work until the stream is done with the call."""
    s = torch.cuda.Stream()
    plain, given = calls(ci8, m, None), calls(ci8, m, s)
    for i in range(len(plain)):
        want = plain[i][0](plain[i][1])
        call, operands = given[i]
        shapes = [(t.shape, t.dtype) for t in operands]
        s.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = call(operands)
        given[i] = None
        del operands
        new = [torch.full(shape, 7, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(2)]
        torch.cuda.current_stream().synchronize()
        s.synchronize()
        del new
        for a, b in zip(*(v if isinstance(v, tuple) else (v,) for v in (want, got))):
            assert torch.equal(a, b), i


def test_a_stream_of_another_device_is_refused(ci8):
    other = SimpleNamespace(device=torch.device("cuda", torch.cuda.current_device() + 1))
    for call, operands in calls(ci8, 4, other):
        with pytest.raises(ValueError, match="stream: on cuda:"):
            call(operands)
