"""Dense products of operands that repeat or overlap their rows, against the
64-bit forms with their counted bounds."""
import math

import pytest
import torch

from tests import dense_reference as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(g, r, c, pitch):
    """[r, c] whose rows are `pitch` elements apart: repeated (0), overlapping, or apart."""
    flat = torch.randn(max(pitch * (r - 1), 0) + c, generator=g, device="cuda").to(BF16)
    return flat.as_strided((r, c), (pitch, 1))


def check_backward(ci8, dy, x, w, label):
    want = ref.linear_backward(dy, x, w)
    for parts in ((True, True, True), (False, True, False), (True, False, False)):
        got = ci8.linear_backward(dy, x, w, need_dx=parts[0], need_dw=parts[1], need_dbias=parts[2])
        torch.cuda.synchronize()
        for name, t, (v, b) in zip(("dx", "dw", "dbias"), got, want):
            if t is not None:
                ref.check(t, v, b, f"{name} {label} {parts}")


@pytest.mark.parametrize("m", [2, 50, 64, 130])
@pytest.mark.parametrize("dy_pitch,x_pitch", [(0, 0), (8, 8), (0, 16), (40, 0), (64, 0), (0, 48)])
def test_backward_repeated_rows(ci8, m, dy_pitch, x_pitch):
    """Row counts below, at and past a stage's 64 rows; both gradients in one launch and alone."""
    print(f"[gpu] backward of repeated rows m={m} dy={dy_pitch} x={x_pitch}", flush=True)
    g = gen(31)
    check_backward(ci8, rows(g, m, 64, dy_pitch), rows(g, m, 48, x_pitch), rows(g, 64, 48, 48), "repeated")


@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64", "128x128d", "256x256/2", "64x64/2"])
@pytest.mark.parametrize("pitch", [0, 8])
def test_backward_repeated_rows_on_every_tile(ci8, monkeypatch, tile, pitch):
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    print(f"[gpu] backward of repeated rows tile={tile} pitch={pitch}", flush=True)
    g = gen(32)
    check_backward(ci8, rows(g, 610, 264, pitch), rows(g, 610, 136, pitch), rows(g, 264, 136, pitch), tile)


@pytest.mark.parametrize("pitch", [0, 8])
def test_infinity_in_a_repeated_operand(ci8, pitch):
    """An infinity meets only its own column's values, none of them zero: the result is the infinity."""
    g = gen(33)
    m, n, k = 50, 64, 48
    dy = rows(g, m, n, 64).abs() + 1
    x = (torch.rand(k + pitch * (m - 1), generator=g, device="cuda").to(BF16) + 1)
    x[-1] = math.inf  # the last column of the last row
    x = x.as_strided((m, k), (pitch, 1))
    dw = ci8.linear_backward(dy, x, torch.ones(n, k, dtype=BF16, device="cuda"))[1]
    assert bool(torch.isfinite(dw[:, :k - 1]).all()) and bool((dw[:, k - 1] == math.inf).all())
    # the same in linear's sum over the rows of a transposed weight, and in dx's over those of w
    w = (torch.rand(k + pitch * (n - 1), generator=g, device="cuda").to(BF16) + 1)
    w[-1] = math.inf
    w = w.as_strided((n, k), (pitch, 1))
    w50 = w[-50:]
    y = ci8.linear(dy[:, :50].contiguous(), w50.t())
    assert bool(torch.isfinite(y[:, :k - 1]).all()) and bool((y[:, k - 1] == math.inf).all())
    dx = ci8.linear_backward(dy[:, :50].contiguous(), torch.ones(m, k, dtype=BF16, device="cuda"), w50)[0]
    assert bool(torch.isfinite(dx[:, :k - 1]).all()) and bool((dx[:, k - 1] == math.inf).all())


@pytest.mark.parametrize("pitch", [0, 8, 48])
def test_linear_overlapping_transposed_weights(ci8, pitch):
    g = gen(34)
    x, w = rows(g, 70, 50, 50), rows(g, 50, 48, pitch).t()
    (v, b), _ = ref.linear(x, w, out_dtype=BF16)
    ref.check(ci8.linear(x, w), v, b, "transposed")
