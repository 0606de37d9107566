"""Plain 64-bit forms of the dense layer and layer norm, and how far a kernel
that sums in 32 bits and rounds once may be from them.

Every function returns (value, bound): |kernel - value| <= bound has to hold
element by element.  The bounds count roundings: a 32-bit operation is off by
2^-24 of its result, a sum of n terms by at most n 2^-24 of the sum of their
magnitudes (2^-23 is used, which also covers a matrix unit that truncates),
and an output's rounding by eps/2 of its value (plus the type's smallest
step, for results below its normal range).
"""
import math

import torch

F32 = 2.0 ** -23
# Activations and slopes come from the hardware's exp2 and reciprocal and the
# math library's erfc, each within a few 2^-24 of its value; an error e of the
# exponent changes the gate p by p (1 - p) e, and |u| p (1 - p) <= 0.28, so the
# value is off by less than 2^-20 |z| and the slope by less than 2^-19.
ACT_ERR, SLOPE_ERR = 2.0 ** -20, 2.0 ** -19
ACT_MAX_SLOPE = 1.13  # the largest |act'| of gelu, its tanh form and silu


def rounding(value, dtype):
    if dtype == torch.float64:
        return torch.zeros_like(value)
    info = torch.finfo(dtype)
    return value.abs() * (info.eps / 2) + info.smallest_normal * info.eps


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + torch.exp(-z))


def slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = 1 / (1 + torch.exp(-c * (z + 0.044715 * z ** 3)))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def linear(x, w, bias=None, activation="none", residual=None, x_scale=None, w_scale=None, out_dtype=None):
    """((y, bound), (z, bound))."""
    integer = x.dtype == torch.int8
    k = x.shape[1]
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    if integer:
        s = torch.ones(z.shape[0], 1, dtype=torch.float64, device=z.device)
        if x_scale is not None:
            s = s * x_scale.double()[:, None]
        if w_scale is not None:
            s = s * w_scale.double()[None, :]
        z = z * s
        err = 3 * F32 * z.abs()  # the integer's conversion, the scales' product, the product with it
    else:
        err = (k + 1) * F32 * (xd.abs() @ wd.abs().t())
    if bias is not None:
        z = z + bias.double()
        err = err + F32 * (z.abs() + err)
    a = act(z, activation)
    aerr = err if activation in ("none", "relu") else ACT_MAX_SLOPE * err + ACT_ERR * z.abs()
    y = a
    if residual is not None:
        y = y + residual.double()
        aerr = aerr + F32 * (y.abs() + aerr)
    return ((y, aerr + rounding(y.abs() + aerr, out_dtype)), (z, err + rounding(z.abs() + err, out_dtype)))


def linear_backward(dy, x, w, z=None, activation="none"):
    """((dx, bound), (dw, bound), (dbias, bound)) with g rounded to the operands' type."""
    dt = dy.dtype
    m, n = dy.shape
    g, gerr = dy.double(), torch.zeros(dy.shape, dtype=torch.float64, device=dy.device)
    if activation != "none":
        exact = activation == "relu"
        s = slope(z.double(), activation)
        gerr = torch.zeros_like(g) if exact else (SLOPE_ERR + F32 * s.abs()) * g.abs()
        g = g * s
    rerr = gerr + (0 if activation in ("none", "relu") else rounding(g.abs() + gerr, dt))
    gm = g.abs() + rerr
    xd, wd = x.double(), w.double()
    dx, dw, db = g @ wd, g.t() @ xd, g.sum(0)
    ex = rerr @ wd.abs() + (n + 1) * F32 * (gm @ wd.abs())
    ew = rerr.t() @ xd.abs() + (m + 1) * F32 * (gm.t() @ xd.abs())
    eb = gerr.sum(0) + (m + 1) * F32 * (g.abs() + gerr).sum(0)
    return ((dx, ex + rounding(dx.abs() + ex, dt)), (dw, ew + rounding(dw.abs() + ew, dt)),
            (db, eb + rounding(db.abs() + eb, dt)))


def _steps(d):
    """Additions one after another in a row's sum: at least 64 threads share a
    row, and their sums are joined in at most 16 + 10 steps."""
    return math.ceil(d / 64) + 26


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """{"y", "mean", "rstd", "top"}: (value, bound) of each; y before its rounding."""
    xd = x.double()
    d = x.shape[1]
    n = _steps(d) * F32
    mean = xd.mean(1)
    emean = n * xd.abs().mean(1) + F32 * mean.abs()
    c = xd - mean[:, None]
    var = c.square().mean(1)
    # the mean's error adds its square to the variance, each value's own rounding twice its relative size
    evar = (n + 4 * F32) * var + 2 * emean * c.abs().mean(1) + emean.square()
    rstd = 1 / torch.sqrt(var + eps)
    erstd = rstd * (0.5 * evar / (var + eps) * (1 + evar / (var + eps)) + 4 * F32)
    w = weight.double() if weight is not None else torch.ones(d, dtype=torch.float64, device=x.device)
    b = bias.double() if bias is not None else torch.zeros(d, dtype=torch.float64, device=x.device)
    y = c * rstd[:, None] * w + b
    ey = w.abs() * (c.abs() * erstd[:, None] + (rstd + erstd)[:, None] * (emean[:, None] + F32 * c.abs())
                    + 2 * F32 * c.abs() * rstd[:, None]) + F32 * (y.abs() + b.abs())
    return {"y": (y, ey), "mean": (mean, emean), "rstd": (rstd, erstd)}


def layer_norm_backward(dy, x, weight, mean, rstd):
    """((dx, bound), (dweight, bound), (dbias, bound)); mean and rstd are taken as given."""
    dt = x.dtype
    m, d = x.shape
    xd, g = x.double(), dy.double()
    mu, r = mean.double()[:, None], rstd.double()[:, None]
    w = weight.double() if weight is not None else torch.ones(d, dtype=torch.float64, device=x.device)
    xh = (xd - mu) * r
    exh = F32 * ((xd.abs() + mu.abs()) * r)  # the difference rounds by what it is taken of at most
    c = g * w
    s1, s2 = c.mean(1, keepdim=True), (c * xh).mean(1, keepdim=True)
    n = (_steps(d) + 4) * F32
    e1 = n * c.abs().mean(1, keepdim=True)
    e2 = n * (c * xh).abs().mean(1, keepdim=True) + (c.abs() * exh).mean(1, keepdim=True)
    dx = r * (c - s1 - xh * s2)
    ex = r * (e1 + xh.abs() * e2 + exh * (s2.abs() + e2) + 4 * F32 * (c.abs() + s1.abs() + (xh * s2).abs()))
    dw, db = (g * xh).sum(0), g.sum(0)
    ew = (m + 2) * F32 * (g * xh).abs().sum(0) + (g.abs() * exh).sum(0)
    eb = (m + 1) * F32 * g.abs().sum(0)
    return tuple((v, e + rounding(v.abs() + e, dt)) for v, e in ((dx, ex), (dw, ew), (db, eb)))


def check(got, value, bound, label):
    assert tuple(got.shape) == tuple(value.shape), (label, tuple(got.shape), tuple(value.shape))
    if not got.numel():
        return
    off = (got.double() - value).abs() - bound
    bad = ~(off <= 0)
    # half a step above the type's largest value, an infinity is the right rounding
    info = torch.finfo(got.dtype)
    edge = info.max * (1 + info.eps / 4)
    inf = torch.isinf(got) & (got.double() * value > 0)
    bad = torch.where(value.abs() - bound > edge, ~inf, bad & ~(inf & (value.abs() + bound >= edge)))
    if bool(bad.any()):
        i = int(torch.where(torch.isnan(off), torch.full_like(off, math.inf), off).reshape(-1).argmax())
        at = [int(v) for v in torch.unravel_index(torch.tensor(i), got.shape)]
        raise AssertionError(f"{label}: {int(bad.sum())} of {got.numel()} values off, worst at {at}: got "
                             f"{float(got.reshape(-1)[i])} want {float(value.reshape(-1)[i])} +- {float(bound.reshape(-1)[i])}")
