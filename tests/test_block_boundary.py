"""The entries around a block in 8-bit floating point on the CPU: bad arguments are
refused on the host before any device is touched, and plans and workspaces are
what the sizes ask for."""
import ctypes

import pytest
import torch

import int8_convolution_forward_amd as ci8
from int8_convolution_forward_amd import dense
from tests.test_dense_boundary import BF16, FAKE, FP16, FP32, I8, NM, NV, mat, size, vec

E4, E5, E8 = 6, 7, 8


def name(code):
    return ci8.STATUS[code]


def quantize(x=mat(64, 300, BF16), q=mat(64, 300, E4), scale=mat(64, 3, E8), qt=NM, st=NM):
    return dense._pack_quantize(*x, *q, *scale, *qt, *st)


def dequantize(q=mat(64, 300, E4), scale=mat(64, 3, E8), x=mat(64, 300, BF16)):
    return dense._pack_dequantize(*q, *scale, *x)


def linear(x=mat(64, 272, E4), w=mat(48, 272, E4), y=mat(64, 48, BF16), residual=NM, preact=NM, xs=mat(64, 3, E8),
           ws=mat(48, 3, E8), bias=NV, act=0):
    return dense._pack_linear_fp8(*x, *w, *y, *residual, *preact, *xs, *ws, *bias, act)


def backward(dy=mat(64, 48, BF16), z=NM, xt=mat(272, 64, E4), xts=mat(272, 1, E8), wt=mat(272, 48, E4), wts=mat(3, 1, E8),
             dx=mat(64, 272, BF16), dw=mat(48, 272, BF16), db=vec(48, BF16), act=0, g=E4):
    return dense._pack_linear_fp8_backward(*dy, *z, *xt, *xts, *wt, *wts, *dx, *dw, *db, act, g)


M8 = mat(8, 40, BF16)


def norm(x=M8, h=M8, r=M8, y=M8, gate=NM, ys=NM, post=NV, weight=NV, bias=NV, mean=NV, rstd=NV, pmean=NV, prstd=NV,
         alpha=1.0, eps=1e-5, kind=0):
    return dense._pack_residual_norm(*x, *h, *r, *y, *gate, *ys, *post, *weight, *bias, *mean, *rstd, *pmean, *prstd, alpha,
                                     eps, kind)


def norm_backward(dr=M8, dy=M8, r=M8, h=M8, dx=M8, dh=M8, gate=NM, dgate=NM, weight=NV, post=NV, mean=vec(8, FP32),
                  rstd=vec(8, FP32), pmean=NV, prstd=NV, dw=vec(40, BF16), db=vec(40, BF16), dp=NV, alpha=1.0, kind=0):
    return dense._pack_residual_norm_backward(*dr, *dy, *r, *h, *dx, *dh, *gate, *dgate, *weight, *post, *mean, *rstd, *pmean,
                                              *prstd, *dw, *db, *dp, alpha, kind)


def clip(a, b=None, max_norm=1.0, norm=FAKE - 256, count=None):
    """(argument, what it points to)."""
    held = [b"".join(dense.struct.pack("=Q2q", *v) for v in t) for t in (a, a if b is None else b)]
    ptrs = [ctypes.cast(ctypes.c_char_p(h), ctypes.c_void_p).value for h in held]
    return dense._pack_clip(*ptrs, len(a) if count is None else count, max_norm, norm), held


def test_structures_match_the_header():
    """The packed sizes are those of the C structures (8-byte members only)."""
    assert len(quantize()) == 8 * 5 * 6
    assert len(dequantize()) == 8 * 3 * 6
    assert len(linear()) == 8 * (7 * 6 + 3 + 1)
    assert len(backward()) == 8 * (8 * 6 + 3 + 2)
    assert len(norm()) == 8 * (6 * 6 + 7 * 3 + 3)
    assert len(norm_backward()) == 8 * (8 * 6 + 9 * 3 + 2)
    assert len(clip([vec(4, FP32)])[0]) == 8 * 5


@pytest.mark.parametrize("over,status", [
    (dict(x=mat(64, 300, I8)), "DTYPE"),
    (dict(x=mat(64, 300, E4)), "DTYPE"),
    (dict(q=mat(64, 300, I8)), "DTYPE"),
    (dict(q=mat(64, 300, E8)), "DTYPE"),
    (dict(q=mat(64, 299, E4)), "OUT_DIMS"),
    (dict(q=mat(64, 300, E4, rs=299)), "STRIDES"),
    (dict(q=mat(64, 300, E4, rs=1, cs=64)), "STRIDES"),
    (dict(scale=mat(64, 2, E8)), "OUT_DIMS"),
    (dict(scale=mat(63, 3, E8)), "OUT_DIMS"),
    (dict(scale=mat(64, 3, FP32)), "DTYPE"),
    (dict(scale=NM), "PARAM"),
    (dict(scale=mat(64, 3, E8, rs=2)), "STRIDES"),
    (dict(x=mat(64, 300, BF16, rs=1, cs=64)), "STRIDES"),
    (dict(q=NM, scale=NM), "NULL"),
    (dict(qt=mat(300, 64, E4)), "PARAM"),
    (dict(qt=mat(300, 63, E4), st=mat(300, 1, E8)), "OUT_DIMS"),
    (dict(qt=mat(300, 64, E5), st=mat(300, 1, E8)), "DTYPE"),
    (dict(qt=mat(300, 64, E4), st=mat(299, 1, E8)), "OUT_DIMS"),
    (dict(q=mat(64, 300, E4, ptr=0)), "NULL"),
    (dict(x=mat(64, 300, FP32, ptr=FAKE + 2)), "PARAM"),
    (dict(x=mat(1 << 30, 1 << 20, BF16), q=mat(1 << 30, 1 << 20, E4), scale=mat(1 << 30, 1 << 13, E8)), "UNSUPPORTED"),
])
def test_quantize_refusals(over, status):
    assert name(dense.lib.dense_quantize(quantize(**over), None)) == "CONV_I8_ERR_" + status


@pytest.mark.parametrize("over,status", [
    (dict(q=mat(64, 300, I8)), "DTYPE"),
    (dict(x=mat(64, 300, E4)), "DTYPE"),
    (dict(x=mat(64, 301, BF16)), "OUT_DIMS"),
    (dict(scale=mat(2, 3, E8)), "OUT_DIMS"),
    (dict(scale=mat(64, 3, BF16)), "DTYPE"),
    (dict(scale=mat(64, 3, E8, rs=1, cs=64)), "STRIDES"),
    (dict(q=mat(64, 300, E4, rs=1, cs=64)), "STRIDES"),
])
def test_dequantize_refusals(over, status):
    assert name(dense.lib.dense_dequantize(dequantize(**over), None)) == "CONV_I8_ERR_" + status


@pytest.mark.parametrize("over,status", [
    (dict(x=mat(64, 272, BF16)), "DTYPE"),
    (dict(x=mat(64, 272, I8)), "DTYPE"),
    (dict(w=mat(48, 272, E5)), "DTYPE"),
    (dict(y=mat(64, 48, E4)), "DTYPE"),
    (dict(w=mat(48, 271, E4)), "CHANNELS"),
    (dict(y=mat(64, 47, BF16)), "OUT_DIMS"),
    (dict(xs=mat(64, 2, E8)), "OUT_DIMS"),
    (dict(xs=mat(1, 3, E8)), "OUT_DIMS"),
    (dict(xs=NM), "DTYPE"),
    (dict(ws=mat(2, 3, E8)), "OUT_DIMS"),
    (dict(ws=mat(48, 3, FP32)), "DTYPE"),
    (dict(ws=mat(48, 3, E8, rs=1, cs=48)), "STRIDES"),
    (dict(ws=mat(48, 3, E8, ptr=0)), "NULL"),
    (dict(residual=mat(64, 48, FP32)), "DTYPE"),
    (dict(preact=mat(64, 47, BF16)), "OUT_DIMS"),
    (dict(preact=mat(64, 48, BF16, rs=40)), "STRIDES"),
    (dict(residual=mat(64, 48, BF16, rs=1, cs=64)), "STRIDES"),
    (dict(bias=vec(47, BF16)), "DIMS"),
    (dict(bias=vec(48, E8)), "DTYPE"),
    (dict(act=5), "PARAM"),
    (dict(x=mat(64, 272, E4, ptr=0)), "NULL"),
    (dict(x=mat(64, 272, E4, rs=-272)), "STRIDES"),
])
def test_linear_fp8_refusals(over, status):
    args = linear(**over)
    want = "CONV_I8_ERR_" + status
    assert size("dense_linear_fp8", args)[0] == want
    assert name(dense.lib.dense_linear_fp8(args, None, 0, None)) == want


@pytest.mark.parametrize("over,status", [
    (dict(dy=mat(64, 48, FP32)), "DTYPE"),
    (dict(g=FP16), "DTYPE"),
    (dict(g=0), "DTYPE"),
    (dict(act=9), "PARAM"),
    (dict(act=256), "PARAM"),
    (dict(act=1), "NULL"),
    (dict(act=1, z=mat(64, 47, BF16)), "DIMS"),
    (dict(act=1, z=mat(64, 48, FP16)), "DTYPE"),
    (dict(dy=mat(64, 48, BF16, rs=1, cs=64)), "STRIDES"),
    (dict(xt=NM), "NULL"),
    (dict(wt=NM), "NULL"),
    (dict(xt=mat(272, 64, E5)), "DTYPE"),
    (dict(xt=mat(272, 63, E4)), "DIMS"),
    (dict(wt=mat(271, 48, E4)), "CHANNELS"),
    (dict(wt=mat(272, 47, E4)), "DIMS"),
    (dict(xts=mat(272, 2, E8)), "OUT_DIMS"),
    (dict(wts=mat(2, 1, E8)), "OUT_DIMS"),
    (dict(dx=mat(63, 272, BF16)), "OUT_DIMS"),
    (dict(dx=mat(64, 272, FP32)), "DTYPE"),
    (dict(dw=mat(48, 271, BF16)), "OUT_DIMS"),
    (dict(dw=mat(48, 272, BF16, rs=8)), "STRIDES"),
    (dict(db=vec(47, BF16)), "DIMS"),
    (dict(db=vec(48, FP32)), "DTYPE"),
])
def test_linear_fp8_backward_refusals(over, status):
    args = backward(**over)
    want = "CONV_I8_ERR_" + status
    assert size("dense_linear_fp8_backward", args)[0] == want
    assert name(dense.lib.dense_linear_fp8_backward(args, None, 0, None)) == want


@pytest.mark.parametrize("over,status", [
    (dict(x=mat(8, 40, E4)), "DTYPE"),
    (dict(h=mat(8, 40, FP16)), "DTYPE"),
    (dict(h=mat(8, 41, BF16)), "DIMS"),
    (dict(h=NM), "PARAM"),                       # r without h
    (dict(h=NM, r=NM, gate=mat(1, 40, BF16)), "PARAM"),
    (dict(h=NM, r=NM, post=vec(40, BF16)), "PARAM"),
    (dict(r=NM), "NULL"),
    (dict(r=mat(8, 39, BF16)), "OUT_DIMS"),
    (dict(r=mat(8, 40, FP32)), "DTYPE"),
    (dict(y=mat(8, 40, FP32)), "DTYPE"),
    (dict(y=NM), "DTYPE"),
    (dict(y=mat(8, 40, E4)), "DTYPE"),           # without scales
    (dict(y=mat(8, 40, E4), ys=mat(8, 2, E8)), "OUT_DIMS"),
    (dict(y=mat(8, 40, E5), ys=mat(8, 1, E8)), "PARAM"),
    (dict(ys=mat(8, 1, E8)), "PARAM"),
    (dict(gate=mat(3, 40, BF16)), "DIMS"),
    (dict(gate=mat(0, 40, BF16)), "DIMS"),
    (dict(gate=mat(16, 40, BF16)), "DIMS"),
    (dict(gate=mat(1, 39, BF16)), "DIMS"),
    (dict(gate=mat(1, 40, FP32)), "DTYPE"),
    (dict(weight=vec(39, BF16)), "DIMS"),
    (dict(bias=vec(40, FP32)), "DTYPE"),
    (dict(post=vec(41, BF16)), "DIMS"),
    (dict(pmean=vec(8, FP32)), "PARAM"),
    (dict(mean=vec(8, BF16)), "DTYPE"),
    (dict(eps=-1.0), "PARAM"),
    (dict(eps=float("nan")), "PARAM"),
    (dict(alpha=float("nan")), "PARAM"),
    (dict(kind=2), "PARAM"),
    (dict(x=mat(8, 40, BF16, rs=1, cs=8)), "STRIDES"),
    (dict(x=mat(8, 0, BF16), h=mat(8, 0, BF16), r=mat(8, 0, BF16), y=mat(8, 0, BF16)), "DIMS"),
])
def test_residual_norm_refusals(over, status):
    assert name(dense.lib.dense_residual_norm(norm(**over), None)) == "CONV_I8_ERR_" + status


@pytest.mark.parametrize("over,status", [
    (dict(r=mat(8, 40, I8)), "DTYPE"),
    (dict(dy=mat(7, 40, BF16)), "DIMS"),
    (dict(dr=mat(8, 40, FP32)), "DTYPE"),
    (dict(dx=mat(8, 41, BF16)), "OUT_DIMS"),
    (dict(dh=NM, gate=mat(1, 40, BF16)), "PARAM"),
    (dict(dh=NM, post=vec(40, BF16)), "PARAM"),
    (dict(h=NM, gate=mat(1, 40, BF16)), "NULL"),
    (dict(dgate=mat(1, 40, BF16)), "PARAM"),
    (dict(gate=mat(2, 40, BF16), dgate=mat(1, 40, BF16)), "OUT_DIMS"),
    (dict(gate=mat(5, 40, BF16)), "DIMS"),
    (dict(mean=NV), "NULL"),
    (dict(rstd=NV), "NULL"),
    (dict(post=vec(40, BF16)), "NULL"),
    (dict(rstd=vec(7, FP32)), "DIMS"),
    (dict(dp=vec(40, BF16)), "PARAM"),
    (dict(dw=vec(40, FP32)), "DTYPE"),
    (dict(db=vec(39, BF16)), "DIMS"),
    (dict(kind=-1), "PARAM"),
])
def test_residual_norm_backward_refusals(over, status):
    args = norm_backward(**over)
    want = "CONV_I8_ERR_" + status
    assert size("dense_residual_norm_backward", args)[0] == want
    assert name(dense.lib.dense_residual_norm_backward(args, None, 0, None)) == want


def wide_backward(m, d, **over):
    """Gradients of the scale alone of m rows of d columns."""
    r = mat(m, d, BF16)
    return norm_backward(**dict(dict(dr=NM, dy=r, r=r, h=NM, dx=r, dh=NM, mean=vec(m, FP32), rstd=vec(m, FP32),
                                     dw=vec(d, BF16), db=NV), **over))


def test_residual_norm_backward_larger_than_a_launch():
    """The sums over rows take a launch of at most 2^32 threads and 65535 jobs."""
    assert size("dense_residual_norm_backward", wide_backward(1, 1 << 25))[0] == "CONV_I8_OK"
    assert size("dense_residual_norm_backward", wide_backward(1, 1 << 26))[0] == "CONV_I8_ERR_UNSUPPORTED"
    assert size("dense_residual_norm_backward", wide_backward(1, 1 << 26, dw=NV))[0] == "CONV_I8_OK"
    # no rows, and the gradients of many rows of the gate to be cleared
    e = mat(0, 40, BF16)
    for gates, want in ((1 << 15, "CONV_I8_OK"), (1 << 16, "CONV_I8_ERR_UNSUPPORTED")):
        gate = mat(gates, 40, BF16)
        args = norm_backward(dr=e, dy=e, r=e, h=e, dx=e, dh=e, gate=gate, dgate=gate, mean=vec(0, FP32), rstd=vec(0, FP32))
        assert size("dense_residual_norm_backward", args)[0] == want


A, B = FAKE, FAKE + (1 << 20)


@pytest.mark.parametrize("a,b,over,status", [
    ([vec(4, I8)], None, {}, "DTYPE"),
    ([NV], None, {}, "DTYPE"),
    ([vec(4, BF16)], [vec(4, FP16)], {}, "DTYPE"),
    ([vec(4, BF16)], [vec(5, BF16)], {}, "OUT_DIMS"),
    ([vec(-1, BF16)], None, {}, "DIMS"),
    ([vec(4, BF16, ptr=0)], None, {}, "NULL"),
    ([vec(4, FP32, ptr=FAKE + 2)], None, {}, "PARAM"),
    ([vec(4, FP32)], None, dict(max_norm=-1.0), "PARAM"),
    ([vec(4, FP32)], None, dict(max_norm=float("nan")), "PARAM"),
    ([vec(4, FP32)], None, dict(norm=0), "NULL"),
    ([vec(4, FP32)], None, dict(count=-1), "DIMS"),
    ([vec(4, FP32), vec(4, FP32)], None, {}, "PARAM"),                                   # one tensor twice, in place
    ([vec(8, FP32, ptr=A), vec(8, FP32, ptr=A + 16)], None, {}, "PARAM"),                # overlapping, in place
    ([vec(8, FP32, ptr=A), vec(8, FP32, ptr=B)], [vec(8, FP32, ptr=B), vec(8, FP32, ptr=A)], {}, "PARAM"),
    ([vec(8, FP32, ptr=A)], [vec(8, FP32, ptr=A + 4)], {}, "PARAM"),                     # into itself, shifted
    ([vec(8, FP32, ptr=A)], None, dict(norm=A + 28), "PARAM"),                           # the norm in a gradient
    ([vec(8, FP32, ptr=A)], [vec(8, FP32, ptr=B)], dict(norm=A), "PARAM"),
    ([vec(8, FP32, ptr=A)], [vec(8, FP32, ptr=B)], dict(norm=A + 32), "OK"),
    ([vec(1 << 40, BF16)] , None, {}, "OK"),
])
def test_clip_refusals(a, b, over, status):
    args, held = clip(a, b, **over)
    want = "CONV_I8_" + ("ERR_" + status if status != "OK" else status)
    assert size("dense_clip_grads", args)[0] == want
    if status != "OK":
        assert name(dense.lib.dense_clip_grads(args, None, 0, None)) == want


def test_clip_takes_one_input_for_two_outputs():
    args, held = clip([vec(8, FP32, ptr=A), vec(8, FP32, ptr=A)], [vec(8, FP32, ptr=B), vec(8, FP32, ptr=B + 32)])
    assert size("dense_clip_grads", args)[0] == "CONV_I8_OK"


def test_null_arguments():
    n = ctypes.c_size_t()
    for e in ("dense_quantize", "dense_dequantize", "dense_residual_norm"):
        assert name(getattr(dense.lib, e)(None, None)) == "CONV_I8_ERR_NULL"
    for e in ("dense_linear_fp8", "dense_linear_fp8_backward", "dense_residual_norm_backward", "dense_clip_grads"):
        assert name(getattr(dense.lib, e)(None, None, 0, None)) == "CONV_I8_ERR_NULL"
        assert name(getattr(dense.lib, e + "_workspace_size")(None, n)) == "CONV_I8_ERR_NULL"


def test_older_entries_refuse_the_new_types():
    from tests import test_dense_boundary as old
    for dt in (E4, E5, E8):
        assert size("dense_linear", old.linear(x=mat(64, 32, dt), w=mat(48, 32, dt)))[0] == "CONV_I8_ERR_DTYPE"
        assert size("dense_linear", old.linear(y=mat(64, 48, dt)))[0] == "CONV_I8_ERR_DTYPE"
        assert size("dense_linear", old.linear(bias=vec(48, dt)))[0] == "CONV_I8_ERR_DTYPE"
        assert size("dense_linear_backward", old.backward(dy=mat(64, 48, dt)))[0] == "CONV_I8_ERR_DTYPE"
        assert name(dense.lib.dense_layer_norm(old.norm(y=mat(8, 32, dt)), None)) == "CONV_I8_ERR_DTYPE"


def test_workspaces_are_checked():
    grads, held = clip([vec(4, FP32)])
    for entry, args in (("dense_linear_fp8", linear(x=mat(64, 273, E4), w=mat(48, 273, E4))),
                        ("dense_linear_fp8_backward", backward()),
                        ("dense_residual_norm_backward", norm_backward()),
                        ("dense_clip_grads", grads)):
        status, need = size(entry, args)
        assert status == "CONV_I8_OK" and need > 0
        for ws, n in ((FAKE, need - 1), (FAKE + 64, need), (None, need)):
            assert getattr(dense.lib, entry)(args, ws, n, None) != 0, entry


def test_empty_problems_are_ok_without_device_work():
    z = lambda r, c, dt: mat(r, c, dt, ptr=0)  # noqa: E731
    assert dense.lib.dense_quantize(quantize(x=z(0, 300, BF16), q=z(0, 300, E4), scale=z(0, 3, E8)), None) == 0
    assert dense.lib.dense_quantize(quantize(x=z(64, 0, BF16), q=z(64, 0, E4), scale=z(64, 0, E8)), None) == 0
    assert dense.lib.dense_dequantize(dequantize(q=z(0, 300, E4), scale=z(0, 3, E8), x=z(0, 300, BF16)), None) == 0
    assert dense.lib.dense_linear_fp8(linear(x=z(0, 272, E4), y=z(0, 48, BF16), xs=z(0, 3, E8)), None, 0, None) == 0
    e = z(0, 40, BF16)
    assert dense.lib.dense_residual_norm(norm(x=e, h=e, r=e, y=e), None) == 0
    assert dense.lib.dense_residual_norm_backward(
        norm_backward(dr=e, dy=e, r=e, h=e, dx=e, dh=e, mean=vec(0, FP32), rstd=vec(0, FP32), dw=NV, db=NV), None, 0, None) == 0


def plan(args):
    buf = ctypes.create_string_buffer(512)
    assert dense.lib.dense_linear_fp8_plan(args, buf, 512) == 0
    return buf.value.decode()


def test_plans(monkeypatch):
    monkeypatch.delenv("CONV_I8_DENSE_TILE", raising=False)
    one = dict(x=mat(1, 272, E4), y=mat(1, 48, BF16), xs=mat(1, 3, E8))
    assert plan(linear(**one)).startswith("kernel=skinny")
    odd = dict(x=mat(1, 273, E4), w=mat(48, 273, E4), y=mat(1, 48, BF16), xs=mat(1, 3, E8))
    assert "a=rows_packed b=rows_packed" in plan(linear(**odd))
    big = dict(x=mat(512, 1024, E4), w=mat(256, 1024, E4), y=mat(512, 256, BF16), xs=mat(512, 8, E8), ws=mat(2, 8, E8))
    assert "a=rows b=rows" in plan(linear(**big)) and "stages=8 " in plan(linear(**big))
    assert "b=rows_packed" in plan(linear(**{**big, "w": mat(256, 1024, E4, rs=1, cs=256)}))
    few = lambda m, n, k, dt=BF16: plan(linear(x=mat(m, k, E4), w=mat(n, k, E4), y=mat(m, n, dt),  # noqa: E731
                                               xs=mat(m, k // 128, E8), ws=mat(n, k // 128, E8)))
    for m, n, k, waves in ((1, 4096, 1024, 4), (4, 8192, 4096, 8), (4, 512, 8192, 16), (16, 4096, 8192, 8),
                           (16, 4112, 8192, 4), (17, 4096, 8192, 4), (32, 4096, 512, 4)):
        assert few(m, n, k) == few(m, n, k, FP32) == f"kernel=skinny waves={waves}"
    assert few(17, 4112, 1024).startswith("kernel=gemm tile") and few(17, 4112, 1024, FP32).startswith("kernel=skinny")
    assert few(33, 512, 1024).startswith("kernel=gemm tile") and few(33, 512, 1024, FP32).startswith("kernel=gemm_bf16")
    for tile, tiles in (("256x256", 2), ("128x128", 8), ("64x64", 32)):
        monkeypatch.setenv("CONV_I8_DENSE_TILE", tile + "/2")
        assert f"tile={tile} tiles={tiles} split=2" in plan(linear(**big))
    monkeypatch.setenv("CONV_I8_DENSE_TILE", "31x7")
    assert size("dense_linear_fp8", linear(**big))[0] == "CONV_I8_ERR_PARAM"
    assert size("dense_linear_fp8_backward", backward())[0] == "CONV_I8_ERR_PARAM"


def test_gradients_take_what_they_need_only():
    assert size("dense_linear_fp8_backward", backward(dw=NM, xt=NM, xts=NM))[0] == "CONV_I8_OK"
    assert size("dense_linear_fp8_backward", backward(dx=NM, wt=NM, wts=NM))[0] == "CONV_I8_OK"
    assert size("dense_linear_fp8_backward", backward(dx=NM, wt=NM, wts=NM, dw=NM, xt=NM, xts=NM))[0] == "CONV_I8_OK"
    assert size("dense_residual_norm_backward", norm_backward(dw=NV, db=NV)) == ("CONV_I8_OK", 0)
    assert size("dense_residual_norm_backward", norm_backward(mean=NV, kind=1))[0] == "CONV_I8_OK"
    assert size("dense_residual_norm_backward", norm_backward(h=NM))[0] == "CONV_I8_OK"


def cpu_calls():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    f = torch.zeros(2, 4)
    return {
        "quantize_fp8": lambda: ci8.quantize_fp8(x),
        "dequantize_fp8": lambda: ci8.dequantize_fp8(q, s),
        "linear_fp8": lambda: ci8.linear_fp8(q, q, s, s),
        "linear_fp8_backward": lambda: ci8.linear_fp8_backward(x, q, s, q, s),
        "residual_norm": lambda: ci8.residual_norm(x, x),
        "residual_norm_fp8": lambda: ci8.residual_norm_fp8(x, x),
        "residual_norm_backward": lambda: ci8.residual_norm_backward(x, x, x, x, f),
        "clip_grad_norm": lambda: ci8.clip_grad_norm([x], 1.0),
    }


@pytest.mark.parametrize("entry", list(cpu_calls()))
def test_wrappers_refuse_host_tensors(entry):
    with pytest.raises(ValueError, match="expected a GPU tensor"):
        cpu_calls()[entry]()


def test_wrappers_refuse_wrong_arguments():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="block: 'columns' is none of rows, tiles"):
        ci8.quantize_fp8(x, block="columns")
    with pytest.raises(ValueError, match="norm: 'group' is none of layer, rms"):
        ci8.residual_norm(x, x, norm="group")
    with pytest.raises(ValueError, match="activation: 'tanh'"):
        ci8.linear_fp8(x, x, x, x, activation="tanh")
    with pytest.raises(ValueError, match="at least one tensor"):
        ci8.clip_grad_norm([], 1.0)
    with pytest.raises(TypeError, match=r"grads\[0\]"):
        ci8.clip_grad_norm([3.0], 1.0)
    with pytest.raises(TypeError):
        ci8.linear_fp8_backward(x, None, None, x, x)
    with pytest.raises(TypeError):
        ci8.residual_norm(None, x)
