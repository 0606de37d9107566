"""Every tile of the dense products with a split inner dimension, in the forward
product and in both gradients; the plan is asked which tile and split ran."""
import math

import pytest
import torch

from tests import dense_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, I8 = torch.bfloat16, torch.float16, torch.int8
TILES = ("256x256", "128x128", "64x64", "128x128d")


@pytest.fixture(scope="module")
def ci8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_convolution_forward_amd as m
    return m


def values(g, *shape, dtype=BF16, scale=1.0):
    if dtype == I8:
        return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(I8)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("split", [2, 3, 7])
@pytest.mark.parametrize("m,n,k", [(2100, 2060, 136), (2049, 2113, 77)])
def test_split_gradients(ci8, monkeypatch, dtype, tile, split, m, n, k):
    """dx sums over n, dw over m: both long enough for the split that is named."""
    print(f"[gpu] linear_backward m={m} n={n} k={k} {dtype} tile={tile} split={split}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(41)
    dy, x, z = values(g, m, n, dtype=dtype, scale=0.5), values(g, m, k, dtype=dtype), values(g, m, n, dtype=dtype)
    w = values(g, n, k, dtype=dtype, scale=1 / math.sqrt(k))
    monkeypatch.setenv("CONV_I8_DENSE_TILE", f"{tile}/{split}")
    plan = ci8.linear_backward_plan(dy, x, w, preact=z, activation="silu")
    assert plan.count(f"tile={tile} ") == 2 and plan.count(f"split={split} ") == 2, plan
    got = ci8.linear_backward(dy, x, w, preact=z, activation="silu")
    torch.cuda.synchronize()
    for name, t, (v, b) in zip(("dx", "dw", "dbias"), got, ref.linear_backward(dy, x, w, z, "silu")):
        ref.check(t, v, b, name)


@pytest.mark.parametrize("dtype", [BF16, I8])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("split", [2, 5])
@pytest.mark.parametrize("m,n,k", [(130, 100, 4096), (33, 257, 3100)])
def test_split_linear(ci8, monkeypatch, dtype, tile, split, m, n, k):
    print(f"[gpu] linear m={m} n={n} k={k} {dtype} tile={tile} split={split}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(42)
    x, w = values(g, m, k, dtype=dtype), values(g, n, k, dtype=dtype, scale=1 / math.sqrt(k))
    b, r = values(g, n), values(g, m, n)
    s = torch.full((m,), 2.0 ** -14, device="cuda") if dtype == I8 else None
    z = torch.empty(m, n, dtype=BF16, device="cuda")
    monkeypatch.setenv("CONV_I8_DENSE_TILE", f"{tile}/{split}")
    plan = ci8.linear_plan(x, w, z)
    assert f"tile={tile} " in plan and f"split={split} " in plan, plan
    y = ci8.linear(x, w, b, activation="gelu", residual=r, x_scale=s, preact=z)
    torch.cuda.synchronize()
    (yv, yb), (zv, zb) = ref.linear(x, w, b, "gelu", r, s, out_dtype=BF16)
    ref.check(y, yv, yb, "y")
    ref.check(z, zv, zb, "z")
