"""CONV_I8_DENSE_TILE on the CPU: the tile and the split that it names are what
runs, and a name that means nothing is refused."""
import pytest
import torch

import int8_convolution_forward_amd as ci8

BF16 = torch.bfloat16
TILES = ("256x256", "128x128", "64x64", "128x128d")


def linear_fields(m, n, k, dtype=BF16):
    return ci8.plan_fields(ci8.linear_plan(torch.zeros(m, k, dtype=dtype), torch.zeros(n, k, dtype=dtype),
                                           torch.zeros(m, n, dtype=BF16)))


@pytest.mark.parametrize("value", ["bogus", "64x64k", "64x6", "128x128dd", "64x64/", "64x64/0", "64x64/-1", "64x64/65",
                                   "64x64/2x", "64x64/2/2", "/2", " 64x64"])
def test_a_name_that_means_nothing_is_refused(monkeypatch, value):
    x, w, o = torch.zeros(4, 64, dtype=BF16), torch.zeros(64, 64, dtype=BF16), torch.zeros(4, 64, dtype=BF16)
    monkeypatch.setenv("CONV_I8_DENSE_TILE", value)
    for call in (lambda: ci8.linear_plan(x, w, o), lambda: ci8.linear_backward_plan(o, x, w)):
        with pytest.raises(ci8.ConvI8Error) as e:
            call()
        assert e.value.name == "CONV_I8_ERR_PARAM"
    monkeypatch.setenv("CONV_I8_DENSE_TILE", "")
    assert "kernel=skinny" in ci8.linear_plan(x, w, o)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("split", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("dtype", [BF16, torch.int8])
def test_the_named_tile_and_split_run(monkeypatch, tile, split, dtype):
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile)
    assert linear_fields(4, 64, 64, dtype)["tile"] == tile
    monkeypatch.setenv("CONV_I8_DENSE_TILE", f"{tile}/{split}")
    f = linear_fields(70, 64, 4096, dtype)
    assert f["tile"] == tile
    stages = int(f["stages"])
    assert stages // 4 >= split
    per = -(-stages // split)  # the parts are equal, so there may be fewer
    assert int(f["split"]) == -(-stages // per) and int(f["per_split"]) == per


@pytest.mark.parametrize("tile", TILES)
def test_a_split_of_too_few_stages_keeps_the_tile(monkeypatch, tile):
    monkeypatch.setenv("CONV_I8_DENSE_TILE", tile + "/7")
    for k, most in ((24, 1), (448, 1), (512, 2), (1088, 4)):
        f = linear_fields(70, 64, k)
        assert f["tile"] == tile and 1 <= int(f["split"]) <= most
    plan = ci8.linear_backward_plan(torch.zeros(520, 264, dtype=BF16), torch.zeros(520, 304, dtype=BF16),
                                    torch.zeros(264, 304, dtype=BF16))
    assert plan.count(f"tile={tile} ") == 2 and "launches=apart" in plan
