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
