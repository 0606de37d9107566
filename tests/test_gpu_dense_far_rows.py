"""Rows millions of elements apart: past the offsets that a tile's loads and
stores hold in 31 bits, operands are copied or read by 64-bit addresses, and
outputs take the row-by-row epilogue."""
import math

import pytest
import torch

from tests import dense_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
OUT = (1 << 20) + 8       # elements: the epilogue's own 31-bit offsets end at rows of 2^20
FAR = (1 << 23) + 16      # rows of one byte and more that a tile does not reach


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def spread(t, pitch):
    """t with its rows `pitch` elements apart (memory between them is not initialised)."""
    r, c = t.shape
    v = torch.empty((r - 1) * pitch + c, dtype=t.dtype, device=t.device).as_strided((r, c), (pitch, 1))
    return v.copy_(t)


def values(g, *shape, dtype=BF16, scale=1.0):
    if dtype == I8:
        return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(I8)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP32), (I8, BF16)])
@pytest.mark.parametrize("m,n,tile", [(3, 72, None), (20, 72, None), (300, 264, None), (300, 264, "256x256"),
                                      (300, 264, "128x128d"), (300, 264, "64x64/2")])
def test_linear_far_outputs(ci8, monkeypatch, dtype, out, m, n, tile):
    """y, residual and preact with rows past the epilogue's tile offsets, whole tiles among them."""
    print(f"[gpu] linear far outputs m={m} n={n} {dtype} tile={tile}", flush=True)
    if tile:
        monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    g = torch.Generator(device="cuda").manual_seed(101)
    k = 1056
    x, w, b = values(g, m, k, dtype=dtype), values(g, n, k, dtype=dtype, scale=1 / math.sqrt(k)), values(g, n, dtype=BF16)
    s = torch.full((m,), 2.0 ** -14, device="cuda") if dtype == I8 else None
    r, y, z = (spread(values(g, m, n, dtype=out), OUT) for _ in range(3))
    (yv, yb), (zv, zb) = ref.linear(x, w, b, "silu", r, s, out_dtype=out)
    ci8.linear(x, w, b, activation="silu", residual=r, x_scale=s, preact=z, out=y)
    torch.cuda.synchronize()
    ref.check(y, yv, yb, "y")
    ref.check(z, zv, zb, "z")


@pytest.mark.parametrize("dtype", [BF16, I8])
@pytest.mark.parametrize("m,n", [(2, 40), (17, 40), (300, 40), (40, 300)])
def test_linear_far_operands(ci8, dtype, m, n):
    """The few-rows kernel's 64-bit form, and copies; the widest buffer passes 2^32 bytes."""
    print(f"[gpu] linear far operands m={m} n={n} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(102)
    x, w = values(g, m, 320, dtype=dtype), values(g, n, 320, dtype=dtype, scale=0.05)
    (v, b), _ = ref.linear(x, w, out_dtype=BF16)
    ref.check(ci8.linear(spread(x, FAR), w), v, b, "far x")
    ref.check(ci8.linear(x, spread(w, FAR)), v, b, "far w")
    if dtype == BF16:
        ref.check(ci8.linear(x, spread(w.t(), (1 << 24) + 8).t()), v, b, "far rows of a transposed w")


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_backward_far_operands(ci8, act):
    print(f"[gpu] linear_backward far operands act={act}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(103)
    m, n, k = 150, 72, 64
    dy, x, w, z = values(g, m, n), values(g, m, k), values(g, n, k), values(g, m, n)
    want = ref.linear_backward(dy, x, w, z, act)
    for far in range(4):
        t = [spread(v, FAR) if i == far else v for i, v in enumerate((dy, x, w, z))]
        got = ci8.linear_backward(t[0], t[1], t[2], preact=t[3], activation=act)
        torch.cuda.synchronize()
        for name, a, (v, b) in zip(("dx", "dw", "dbias"), got, want):
            ref.check(a, v, b, f"{name} far={far}")


@pytest.mark.parametrize("d", [5, 96, 3001, 20000, 66000])
def test_norm_far_rows(ci8, d):
    """Rows 2^29 elements apart, gigabytes from the first to the last."""
    print(f"[gpu] layer norm far rows d={d}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(104)
    x, dy = values(g, 6, d), values(g, 6, d)
    far, fdy = spread(x, 1 << 29), spread(dy, 1 << 29)
    got, want = ci8.layer_norm(far), ci8.layer_norm(x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(ci8.layer_norm_i8(far), ci8.layer_norm_i8(x)))
    a = ci8.layer_norm_backward(fdy, far, None, *want[1:])
    b = ci8.layer_norm_backward(dy, x, None, *want[1:])
    assert all(torch.equal(p, q) for p, q in zip(a, b))
