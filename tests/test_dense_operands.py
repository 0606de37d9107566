"""Which operands of the dense products are read in place, on the CPU: the
product kernel ends a columns-form operand by the byte range of its last inner
row, which hides the inner rows past the end only where rows do not overlap."""
import pytest
import torch

import int8_convolution_forward_amd as ci8

BF16 = torch.bfloat16


def backward_plan(dy, x, w, **kw):
    head, rest = ci8.linear_backward_plan(dy, x, w, **kw).split(" dx: ")
    dx, dw = rest.split("; dw: ")
    return ci8.plan_fields(head), ci8.plan_fields(dx), ci8.plan_fields(dw)


def rows(r, c, pitch):
    """[r, c] whose rows are `pitch` elements apart, fewer than c where they overlap."""
    return torch.zeros(max(pitch * (r - 1), 0) + c, dtype=BF16).as_strided((r, c), (pitch, 1))


@pytest.mark.parametrize("pitch", [0, 8, 40])
def test_overlapping_rows_are_copied_for_the_weight_gradient(pitch):
    """dw sums over the rows of dy and x, both of 48 and more columns."""
    w = torch.zeros(64, 48, dtype=BF16)
    head, dx, dw = backward_plan(rows(50, 64, pitch), rows(50, 48, pitch), w)
    assert head["g"] == "written" and dw["b"] == "cols_packed"
    head, _, dw = backward_plan(rows(50, 64, 64), rows(50, 48, 48), w)
    assert head["g"] == "dy" and dw["b"] == "cols"
    head, _, dw = backward_plan(rows(1, 64, 64), rows(1, 48, 48), w)  # one row overlaps nothing
    assert head["g"] == "dy" and dw["b"] == "cols"
    # without dw only dx = g w reads dy, by rows
    assert backward_plan(rows(50, 64, pitch), rows(50, 48, 48), w, need_dw=False)[0]["g"] == "dy"


@pytest.mark.parametrize("pitch", [0, 8, 40])
def test_overlapping_weights_are_copied(pitch):
    """dx sums over the rows of w, and linear over the rows of a transposed one."""
    w = rows(64, 48, pitch)
    _, dx, _ = backward_plan(rows(50, 64, 64), rows(50, 48, 48), w)
    assert dx["b"] == "cols_packed"
    x, out = rows(50, 64, 64), rows(50, 48, 48)
    plan = ci8.plan_fields(ci8.linear_plan(x, w.t(), out))
    assert plan["b"] == "cols_packed"
    assert ci8.plan_fields(ci8.linear_plan(x, rows(64, 48, 48).t(), out))["b"] == "cols"


def far_rows(r, c, pitch, dtype=3):
    from int8_convolution_forward_amd import dense
    return (0x1000000, r, c, pitch, 1, dtype), dense


@pytest.mark.parametrize("pitch", [1 << 23, 1 << 26, 1 << 30])
def test_rows_out_of_a_tiles_reach_are_copied(pitch):
    """Offsets inside a tile are 31-bit: rows further apart than that are copied, not refused."""
    import ctypes
    x, dense = far_rows(64, 32, pitch)
    w, y = far_rows(48, 32, pitch)[0], far_rows(64, 48, pitch)[0]
    buf = ctypes.create_string_buffer(512)
    assert dense.lib.dense_linear_plan(dense._pack_linear(*x, *w, *y, *dense._NO_MAT, *dense._NO_MAT, *dense._NO_VEC,
                                                          *dense._NO_VEC, *dense._NO_VEC, 0), buf, 512) == 0
    plan = ci8.plan_fields(buf.value.decode())
    assert plan["a"] == "rows_packed" and plan["b"] == "rows_packed"
    dx, dw = far_rows(64, 32, 32)[0], far_rows(48, 32, 32)[0]
    args = dense._pack_linear_backward(*y, *x, *w, *dense._NO_MAT, *dx, *dw, *dense._NO_VEC, 0)
    assert dense.lib.dense_linear_backward_plan(args, buf, 512) == 0
    text = buf.value.decode()
    assert text.startswith("g=written") and text.count("b=cols_packed") == (2 if pitch * 2 > (1 << 31) // 64 else 0)
