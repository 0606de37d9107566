"""Plain 64-bit forms of the operators around a block in 8-bit floating point,
and how far a kernel that works in 32 bits and rounds once may be from them.

As in tests/dense_reference.py a function returns (value, bound) pairs; F32
counts a 32-bit operation.  Where a quantised value depends on 32-bit work, its
bound covers every value that the rounding of a number within that work's error can
give.
"""
import math

import torch

from tests.dense_reference import ACT_ERR, ACT_MAX_SLOPE, F32, SLOPE_ERR, act, rounding, slope, _steps

BLOCK = 128
# bits of the mantissa, exponent of the least normal value, exponent of the largest value (1.75 times that power)
FORMATS = {torch.float8_e4m3fn: (3, -6, 8), torch.float8_e5m2: (2, -14, 15)}


def pow2(e):
    """2^e in 64 bits from its bits (torch's ldexp and exp2 are off by a rounding on some devices)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def blocks(n):
    return -(-n // BLOCK)


def block_max(x, tiles):
    """Largest finite magnitude of each block, [rows or rows of tiles, blocks of a row]."""
    m, k = x.shape
    h = BLOCK if tiles else 1
    a = x.abs()
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a))
    a = torch.nn.functional.pad(a, (0, -k % BLOCK, 0, -m % h))
    return a.reshape(a.shape[0] // h, h, blocks(k), BLOCK).amax((1, 3))


def exponents(top, dtype):
    """The least e >= -127 with top 2^-e <= 1.75 2^emax."""
    part, e = torch.frexp(top.double())
    e = e - 1 - FORMATS[dtype][2] + (part > 0.875)
    return torch.where(top > 0, e, torch.full_like(e, -127)).clamp_min(-127)


def spread(e, shape, tiles):
    """A block's number for each of its values."""
    if tiles:
        e = e.repeat_interleave(BLOCK, 0)[:shape[0]]
    return e.repeat_interleave(BLOCK, 1)[:, :shape[1]]


def rounded(x, e, dtype):
    """x rounded to multiples of what the format resolves with a scale of 2^e, half to even (x in 64 bits)."""
    bits, least, _ = FORMATS[dtype]
    v = x * pow2(-e)
    _, p = torch.frexp(v)
    step = pow2((p - 1).clamp_min(least) - bits)
    q = torch.round(v / step) * step
    q = torch.where(torch.isfinite(x), q, torch.full_like(q, math.nan))
    return q * pow2(e)


def quantized(x, tiles, dtype):
    """(values, exponents of the blocks)."""
    x = x.double()
    e = exponents(block_max(x, tiles), dtype)
    return rounded(x, spread(e, x.shape, tiles), dtype), e


def quantized_within(x, err, dtype):
    """(values, bound): rows of x quantised where x is known to within err."""
    x, err = x.double(), torch.as_tensor(err, dtype=torch.float64, device=x.device).expand(x.shape)
    value, _ = quantized(x, False, dtype)
    top = block_max(x, False)
    slack = block_max(err, False)
    bound = torch.zeros_like(value)
    for t in (top - slack, top + slack):
        e = spread(exponents(t.clamp_min(0), dtype), x.shape, False)
        for v in (x - err, x + err):
            bound = torch.maximum(bound, (rounded(v, e, dtype) - value).abs())
    return value, bound


def values(q, scale):
    """What (q, e8m0 scale) stand for."""
    m, k = q.shape
    tiles = scale.shape[0] != m
    e = scale.view(torch.uint8).to(torch.int32) - 127
    return q.float().double() * pow2(spread(e, (m, k), tiles))


def cut(a, b):
    """What the matrix unit may cut off sums over k of products a[m, k] b[n, k] of 8-bit values: of each eight
    consecutive products, the largest at least has all its bits, and the others lose less than 2^-13 of a number
    that is no larger than it."""
    k = a.shape[1]
    pad = lambda t: torch.nn.functional.pad(t.abs(), (0, -k % 8)).reshape(t.shape[0], -1, 8)  # noqa: E731
    a, b = pad(a), pad(b)
    most = [torch.zeros(0, b.shape[0], dtype=torch.float64, device=a.device)]
    step = max(1, (1 << 25) // max(1, b.numel()))
    for i in range(0, a.shape[0], step):
        top = (a[i:i + step, None] * b[None]).amax(3) if k else a.new_zeros(min(step, a.shape[0] - i), b.shape[0], 1)
        most.append(7 * 2.0 ** -13 * top.sum(2))
    return torch.cat(most)


def linear(x, x_scale, w, w_scale, bias=None, activation="none", residual=None, out_dtype=torch.bfloat16):
    """((y, bound), (z, bound))."""
    xd, wd = values(x, x_scale), values(w, w_scale)
    k = x.shape[1]
    z = xd @ wd.t()
    err = (k + 1) * F32 * (xd.abs() @ wd.abs().t())
    if out_dtype != torch.float32:
        err = err + cut(xd, wd)
    if bias is not None:
        z = z + bias.double()
        err = err + F32 * (z.abs() + err)
    y = act(z, activation)
    yerr = err if activation in ("none", "relu") else ACT_MAX_SLOPE * err + ACT_ERR * z.abs()
    if residual is not None:
        y = y + residual.double()
        yerr = yerr + F32 * (y.abs() + yerr)
    return ((y, yerr + rounding(y.abs() + yerr, out_dtype)), (z, err + rounding(z.abs() + err, out_dtype)))


def linear_backward(dy, xt, xt_scale, wt, wt_scale, z=None, activation="none", g_dtype=torch.float8_e4m3fn):
    """((dx, bound), (dw, bound), (dbias, bound))."""
    dt = dy.dtype
    m, n = dy.shape
    g, gerr = dy.double(), torch.zeros(dy.shape, dtype=torch.float64, device=dy.device)
    if activation != "none":
        s = slope(z.double(), activation)
        gerr = torch.zeros_like(g) if activation == "relu" else (SLOPE_ERR + F32 * s.abs()) * g.abs()
        g = g * s
    out = []
    for q, qerr, w, inner in ((*quantized_within(g, gerr, g_dtype), values(wt, wt_scale), n),
                              (*quantized_within(g.t().contiguous(), gerr.t().contiguous(), g_dtype),
                               values(xt, xt_scale), m)):
        v = q @ w.t()
        e = qerr @ w.abs().t() + (inner + 1) * F32 * ((q.abs() + qerr) @ w.abs().t()) + cut(q.abs() + qerr, w)
        out.append((v, e + rounding(v.abs() + e, dt)))
    db = g.sum(0)
    eb = gerr.sum(0) + (m + 1) * F32 * (g.abs() + gerr).sum(0)
    return out[0], out[1], (db, eb + rounding(db.abs() + eb, dt))


def norm(x, weight, bias, kind, eps=1e-5):
    """{"y", "mean", "rstd"}: (value, bound) of the norm of x's rows, y before its rounding; see
    dense_reference.layer_norm."""
    xd = x.double()
    d = x.shape[1]
    n = _steps(d) * F32
    zero = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    mean = xd.mean(1) if kind == "layer" else zero
    emean = n * xd.abs().mean(1) + F32 * mean.abs() if kind == "layer" else zero
    c = xd - mean[:, None]
    var = c.square().mean(1)
    evar = (n + 4 * F32) * var + 2 * emean * c.abs().mean(1) + emean.square()
    rstd = 1 / torch.sqrt(var + eps)
    erstd = rstd * (0.5 * evar / (var + eps) * (1 + evar / (var + eps)) + 4 * F32)
    w = weight.double() if weight is not None else torch.ones(d, dtype=torch.float64, device=x.device)
    b = bias.double() if bias is not None else torch.zeros(d, dtype=torch.float64, device=x.device)
    y = c * rstd[:, None] * w + b
    ey = w.abs() * (c.abs() * erstd[:, None] + (rstd + erstd)[:, None] * (emean[:, None] + F32 * c.abs())
                    + 2 * F32 * c.abs() * rstd[:, None]) + F32 * (y.abs() + b.abs())
    return {"y": (y, ey), "mean": (mean, emean), "rstd": (rstd, erstd)}


def each_row(gate, m):
    """The gate of every row."""
    g = gate.double().reshape(-1, gate.shape[-1])
    return g.repeat_interleave(m // g.shape[0], 0)


def residual(x, h, gate, post_weight, scale, kind, eps=1e-5):
    """(r, bound) before its rounding."""
    n, en = h.double(), torch.zeros(h.shape, dtype=torch.float64, device=h.device)
    if post_weight is not None:
        n, en = norm(h, post_weight, None, kind, eps)["y"]
    if gate is not None:
        g = each_row(gate, x.shape[0])
        n, en = n * g, en * g.abs() + F32 * (n * g).abs()
    alpha = float(torch.tensor(scale, dtype=torch.float32))
    s = alpha * x.double()
    return s + n, en + F32 * (s.abs() + (s + n).abs() + n.abs())


def _norm_gradient(dy, edy, x, weight, mean, rstd, kind):
    """(gradient by x, bound, normed x, bound) from a gradient known to within edy."""
    d = x.shape[1]
    xd, r = x.double(), rstd.double()[:, None]
    mu = mean.double()[:, None] if kind == "layer" else torch.zeros_like(r)
    w = weight.double() if weight is not None else torch.ones(d, dtype=torch.float64, device=x.device)
    xh = (xd - mu) * r
    exh = 2 * F32 * ((xd.abs() + mu.abs()) * r)
    c = dy * w
    ec = edy * w.abs() + F32 * c.abs()
    n = (_steps(d) + 4) * F32
    s2 = (c * xh).mean(1, keepdim=True)
    e2 = n * ((c.abs() + ec) * (xh.abs() + exh)).mean(1, keepdim=True) + (ec * xh.abs() + (c.abs() + ec) * exh).mean(1, keepdim=True)
    if kind == "layer":
        s1 = c.mean(1, keepdim=True)
        e1 = n * (c.abs() + ec).mean(1, keepdim=True) + ec.mean(1, keepdim=True)
    else:
        s1 = e1 = torch.zeros_like(s2)
    dx = r * (c - s1 - xh * s2)
    ex = r * (ec + e1 + xh.abs() * e2 + exh * (s2.abs() + e2) + 4 * F32 * (c.abs() + s1.abs() + (xh * s2).abs()))
    return dx, ex, xh, exh


def residual_backward(dr, dy, r, h, stats, weight, gate, post_weight, scale, kind):
    """{name: (value, bound)}; the statistics are taken as given."""
    dt = r.dtype
    m, d = r.shape
    zero = torch.zeros(m, d, dtype=torch.float64, device=r.device)
    g = dy.double()
    t, et, rh, erh = _norm_gradient(g, zero, r, weight, stats[0], stats[1], kind)
    if dr is not None:
        t = t + dr.double()
        et = et + F32 * (t.abs() + et)
    alpha = float(torch.tensor(scale, dtype=torch.float32))

    def summed(v, e, groups=1):
        """Sums over the rows of each group, of values known to within e."""
        each = m // groups if groups else 0
        v, e = (u.reshape(groups, each, d) for u in (v, e))
        return v.sum(1), e.sum(1) + (each + 2) * F32 * (v.abs() + e).sum(1)

    out = {"dx": (alpha * t, abs(alpha) * et + F32 * (alpha * t).abs())}
    one = lambda p: (p[0][0], p[1][0])  # noqa: E731
    out["dweight"] = one(summed(g * rh, g.abs() * erh + F32 * (g * rh).abs()))
    out["dbias"] = one(summed(g, zero))
    if h is not None:
        n, en, hh, ehh = h.double(), zero, None, None
        if post_weight is not None:
            mean, rstd = stats[2].double()[:, None], stats[3].double()[:, None]
            if kind != "layer":
                mean = torch.zeros_like(rstd)
            hh = (n - mean) * rstd
            ehh = 2 * F32 * (n.abs() + mean.abs()) * rstd
            pw = post_weight.double()
            n, en = hh * pw, ehh * pw.abs() + F32 * (hh * pw).abs()
        u, eu = t, et
        if gate is not None:
            groups = gate.reshape(-1, d).shape[0]
            v, e = summed(t * n, et * (n.abs() + en) + t.abs() * en + F32 * (t * n).abs(), groups)
            out["dgate"] = v.reshape(gate.shape), e.reshape(gate.shape)
            gr = each_row(gate, m)
            u, eu = t * gr, et * gr.abs() + F32 * (t * gr).abs()
        if post_weight is not None:
            out["dpost_weight"] = one(summed(u * hh, eu * (hh.abs() + ehh) + u.abs() * ehh + F32 * (u * hh).abs()))
            u, eu, _, _ = _norm_gradient(u, eu, h, post_weight, stats[2], stats[3], kind)
        out["dh"] = (u, eu)
    return {k: (v, e + rounding(v.abs() + e, dt)) for k, (v, e) in out.items()}
