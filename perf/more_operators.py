"""Measured cases of the operators around a block in 8-bit floating point: the
quantiser, the dense layer on its values and scales with the gradients, the norm
fused with a residual connection and its gradients, and the clipping of gradients
by their global norm.

`run` computes a case with plain torch operations in 32 bits, or, where `own`
is true, with the library's kernels.  `exact` computes the same outputs in 64
bits from the definitions:

    quantize_fp8            a scale 2^e for each block (128 values of a row, or 128 x 128), e the least with
                            max |x| 2^-e no more than the format's largest value; q = round(x 2^-e), half to even
    linear_fp8              z = sum over k of (q_x scale_x)(q_w scale_w) + bias;  y = act(z) + residual
    linear_fp8_backward     g = dy * act'(z);  dx = Q(g) w;  dw = Q(g^T) x;  dbias = sum over rows of g
                            Q: rows of its argument quantised as above and taken back
    residual_norm           n = norm(h) * post_weight, or h;  r = scale * x + gate * n;  y = norm(r) * weight + bias
    residual_norm_backward  the gradients of it from those of r and y
    clip_grad_norm          norm of all gradients together; gradients * min(1, max_norm / norm)

Values held in 8 bits are returned as the numbers that they stand for, by the
library's own dequantize_fp8 where `own` is true.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
BLOCK = 128
_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_MANTISSA = {"e4m3": (3, -6, 8), "e5m2": (2, -14, 15)}  # bits, least normal exponent, exponent of the largest value
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _quantize(name, dtype, form, block, transposed, m, k):
    return {"name": name, "op": "quantize", "dtype": dtype, "format": form, "block": block, "transposed": transposed,
            "m": m, "k": k}


def _linear(name, out, m, n, k, act, residual, keep):
    return {"name": name, "op": "linear", "out": out, "m": m, "n": n, "k": k, "act": act, "residual": residual,
            "keep": keep}


def _linear_backward(name, dtype, form, m, n, k, act):
    return {"name": name, "op": "linear_backward", "dtype": dtype, "format": form, "m": m, "n": n, "k": k, "act": act}


def _norm(name, dtype, norm, out, gate, post, m, d):
    return {"name": name, "op": "norm", "dtype": dtype, "norm": norm, "out": out, "gate": gate, "post": post, "m": m,
            "d": d}


def _norm_backward(name, dtype, norm, gate, post, m, d):
    return {"name": name, "op": "norm_backward", "dtype": dtype, "norm": norm, "gate": gate, "post": post, "m": m, "d": d}


def _clip(name, dtype, tensors, width, clips):
    return {"name": name, "op": "clip", "dtype": dtype, "tensors": tensors, "width": width, "clips": clips}


def listed():
    return [
        # a small ragged batch's activations, with the transposed copy that the weight gradient takes
        _quantize("quantize_ragged_fp16", "fp16", "e4m3", "rows", True, 777, 1032),
        # a training batch's activations between two products, both copies
        _quantize("quantize_train_bf16", "bf16", "e4m3", "rows", True, 8192, 8192),
        # one token through the widening product of a feed-forward block: latency and weight traffic
        _linear("linear_token", "bf16", 1, 8192, 2048, "gelu_tanh", False, False),
        # a prompt through the widening product
        _linear("linear_prompt", "bf16", 4096, 8192, 2048, "gelu_tanh", False, False),
        # gradients of a small ragged batch
        _linear_backward("linear_backward_ragged_fp16", "fp16", "e5m2", 777, 1032, 520, "silu"),
        # gradients of a training step's product
        _linear_backward("linear_backward_train_bf16", "bf16", "e4m3", 8192, 8192, 2048, "gelu_tanh"),
        # the norm between two blocks for a few tokens (decoding)
        _norm("norm_tokens_bf16", "bf16", "rms", "same", "none", False, 4, 2048),
        # a training batch of sequences that each have a gate, with a norm after the block as well
        _norm("norm_train_bf16", "bf16", "layer", "same", "sequences", True, 16384, 4096),
        # its gradients: an odd width in 32 bits with one gate for all rows, and the training batch
        _norm_backward("norm_backward_odd_fp32", "fp32", "rms", "vector", False, 1003, 1537),
        _norm_backward("norm_backward_train_bf16", "bf16", "layer", "sequences", True, 16384, 4096),
        # gradients of one small layer's parameters, within the limit
        _clip("clip_layer_fp32", "fp32", 6, 256, False),
        # gradients of several layers in 16 bits, above the limit, into the buffers that the update reads
        _clip("clip_model_bf16", "bf16", 48, 2048, True),
    ]


def _log_size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; four in ten are left as
    drawn (odd ones among them), the others are rounded to what models use."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    step = rng.choice((1, 1, 8, 16, 64))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "linear_backward", "norm", "norm_backward", "clip"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "quantize":
        m, k = _log_size(rng, 1, 16384), _log_size(rng, 64, 16384)
        while m * k > 1 << 26:  # the largest listed one
            m = max(1, m // 2)
        case = _quantize("", dtype, rng.choice(("e4m3", "e4m3", "e5m2")), rng.choice(("rows", "tiles")),
                         rng.random() < 0.5, m, k)
    elif op in ("linear", "linear_backward"):
        m, n, k = _log_size(rng, 1, 8192), _log_size(rng, 64, 8192), _log_size(rng, 64, 8192)
        most = 1 << (36 if op == "linear" else 37)  # the largest listed product
        while m * n * k > most:
            m = max(1, m // 2)
        act = rng.choice(ACTS)
        if op == "linear":
            case = _linear("", rng.choice(("bf16", "bf16", "fp16", "fp32")), m, n, k, act, rng.random() < 0.5,
                           rng.random() < 0.3)
        else:
            case = _linear_backward("", rng.choice(("bf16", "fp16")), rng.choice(("e4m3", "e5m2")), m, n, k, act)
    elif op in ("norm", "norm_backward"):
        m, d = _log_size(rng, 1, 16384), _log_size(rng, 64, 16384)
        while m * d > 1 << 26:  # the largest listed norm
            m = max(1, m // 2)
        kind, gate, post = rng.choice(("rms", "layer")), rng.choice(("none", "vector", "sequences")), rng.random() < 0.5
        if op == "norm":
            case = _norm("", dtype, kind, rng.choice(("same", "same", "fp8")), gate, post, m, d)
        else:
            case = _norm_backward("", dtype, kind, gate, post, m, d)
    else:
        case = _clip("", dtype, rng.choice((1, 3, 12, 40)), _log_size(rng, 32, 2048), rng.random() < 0.5)
    del case["name"]
    return case


def _normal(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _activations(gen, m, k, dtype=torch.float32):
    """Unit-variance values with a few channels an order of magnitude larger,
    as residual streams have."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    loud = torch.rand(k, generator=gen, device="cuda") < 0.01
    return (x * torch.where(loud, 8.0, 1.0)).to(dtype)


def _sequences(m):
    """Sequences of a batch of m rows: 8 or 4 or 2 of one length where that divides it."""
    return next(g for g in (8, 4, 2, 1) if m % g == 0)


def _shapes(tensors, width):
    """Parameters as a stack of feed-forward layers has them: two matrices and four vectors each, the last cut short."""
    layer = [(4 * width, width), (4 * width,), (width, 4 * width), (width,), (width,), (width,)]
    return [layer[i % 6] for i in range(tensors)]


def _blocks(x, block):
    """x padded with zeros to whole blocks of 128 values of a row ("rows") or 128 x 128 ("tiles"), as
    [rows of blocks, rows in one, blocks of a row, 128]."""
    h = BLOCK if block == "tiles" else 1
    m, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % BLOCK, 0, -m % h))
    return x.reshape(x.shape[0] // h, h, x.shape[1] // BLOCK, BLOCK)


def _spread(scale, block, m, k):
    """A scale for every value from one for every block."""
    if block == "tiles":
        scale = scale.repeat_interleave(BLOCK, 0)[:m]
    return scale.repeat_interleave(BLOCK, 1)[:, :k]


def _scales(x, block, form):
    """Exponents of the blocks' scales, in x's precision."""
    top = _blocks(x.abs(), block).amax((1, 3))
    part, exp = torch.frexp(top)  # top = part 2^exp, part in [1/2, 1)
    e = exp - 1 - _MANTISSA[form][2] + (part > 0.875)
    return torch.where(top > 0, e, -127).clamp_min(-127)


def _encode(x, block, form):
    """(q, e8m0 scales) of a 32-bit x."""
    e = _scales(x, block, form)
    q = torch.ldexp(x, -_spread(e, block, *x.shape)).to(_FORMATS[form])
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _decode(q, scale, block):
    """The values of (q, e8m0 scales), in 32 bits."""
    e = scale.view(torch.uint8).to(torch.int32) - 127
    return torch.ldexp(q.float(), _spread(e, block, *q.shape))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        s["x"] = _activations(gen, case["m"], case["k"], _DTYPES[case["dtype"]])
    elif case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        wide = _DTYPES[case["out"]]
        s["x"], s["x_scale"] = _encode(_activations(gen, m, k), "rows", "e4m3")
        s["w"], s["w_scale"] = _encode(_normal(gen, n, k, scale=1 / math.sqrt(k)), "tiles", "e4m3")
        s["bias"] = _normal(gen, n, dtype=wide, scale=0.5)
        if case["residual"]:
            s["res"] = _activations(gen, m, n, wide)
    elif case["op"] == "linear_backward":
        m, n, k = case["m"], case["n"], case["k"]
        dtype = _DTYPES[case["dtype"]]
        # what the forward pass left: both operands transposed
        s["xt"], s["xt_scale"] = _encode(_activations(gen, m, k).t().contiguous(), "rows", "e4m3")
        s["wt"], s["wt_scale"] = _encode(_normal(gen, k, n, scale=1 / math.sqrt(k)), "tiles", "e4m3")
        s["dy"] = _normal(gen, m, n, dtype=dtype, scale=0.1)
        s["z"] = _normal(gen, m, n, dtype=dtype) if case["act"] != "none" else None
    elif case["op"] in ("norm", "norm_backward"):
        m, d = case["m"], case["d"]
        dtype = _DTYPES[case["dtype"]]
        s["scale"] = 0.8
        s["weight"] = _normal(gen, d, scale=0.2).add_(1).to(dtype)
        s["bias"] = _normal(gen, d, dtype=dtype, scale=0.2)
        s["post_weight"] = _normal(gen, d, scale=0.2).add_(1).to(dtype) if case["post"] else None
        s["gate"] = None
        if case["gate"] != "none":
            shape = (d,) if case["gate"] == "vector" else (_sequences(m), d)
            s["gate"] = _normal(gen, *shape, dtype=dtype, scale=0.5)
        s["h"] = (_normal(gen, m, d) * 0.7 + _normal(gen, m, 1, scale=0.3)).to(dtype)
        if case["op"] == "norm":
            s["x"] = (_normal(gen, m, d) * 1.5 + _normal(gen, m, 1)).to(dtype)
        else:
            # what the forward pass left: the sum r and the statistics of both norms
            s["r"] = (_normal(gen, m, d) * 1.5 + _normal(gen, m, 1)).to(dtype)
            s["stats"] = torch.cat([_stats(t.float(), case["norm"]) for t in ((s["r"], s["h"]) if case["post"] else (s["r"],))])
            s["dr"], s["dy"] = _normal(gen, m, d, dtype=dtype, scale=0.1), _normal(gen, m, d, dtype=dtype, scale=0.1)
    else:
        shapes = _shapes(case["tensors"], case["width"])
        s["grads"] = [_normal(gen, *shape, dtype=_DTYPES[case["dtype"]], scale=0.01) for shape in shapes]
        norm = 0.01 * math.sqrt(sum(math.prod(shape) for shape in shapes))
        s["max_norm"] = norm / 4 if case["clips"] else norm * 4
        # buffers of the update, or none: in place, where gradients within the limit stay as they are
        s["out"] = [torch.empty_like(g) for g in s["grads"]] if case["clips"] else None
    return s


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def _stats(x, norm):
    """Mean (0 for the root mean square) and 1 / sqrt(mean square distance from it + eps) of each row: [2, rows]."""
    mean = x.mean(1) if norm == "layer" else torch.zeros_like(x[:, 0])
    return torch.stack([mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)])


def _gate_rows(s, m):
    """The gate of every row, and how many rows share one."""
    gate = s["gate"].float().reshape(-1, s["gate"].shape[-1])
    each = m // gate.shape[0]
    return gate.repeat_interleave(each, 0), each


def _norm_gradient(dy, x, weight, stats, norm):
    """(gradient of x, normed x) of norm(x) * weight."""
    xh = (x - stats[0][:, None]) * stats[1][:, None]
    c = dy * weight
    middle = c.mean(1, keepdim=True) if norm == "layer" else 0
    return stats[1][:, None] * (c - middle - xh * (c * xh).mean(1, keepdim=True)), xh


def _plain(s):
    if s["op"] == "quantize":
        x = s["x"].float()
        # 8-bit values times a power of two: they are numbers of 16 bits exactly
        out = {"x": _decode(*_encode(x, s["block"], s["format"]), s["block"]).to(torch.bfloat16)}
        if s["transposed"]:
            out["xt"] = _decode(*_encode(x.t(), s["block"], s["format"]), s["block"]).to(torch.bfloat16)
        return out
    if s["op"] == "linear":
        dtype = _DTYPES[s["out"]]
        z = _decode(s["x"], s["x_scale"], "rows") @ _decode(s["w"], s["w_scale"], "tiles").t() + s["bias"].float()
        y = _act(z, s["act"])
        if s["residual"]:
            y = y + s["res"].float()
        out = {"y": y.to(dtype)}
        if s["keep"]:
            out["z"] = z.to(dtype)
        return out
    if s["op"] == "linear_backward":
        dtype, form = _DTYPES[s["dtype"]], s["format"]
        g = s["dy"].float()
        if s["act"] != "none":
            g = g * _act_slope(s["z"].float(), s["act"])
        dx = _decode(*_encode(g, "rows", form), "rows") @ _decode(s["wt"], s["wt_scale"], "tiles").t()
        dw = _decode(*_encode(g.t(), "rows", form), "rows") @ _decode(s["xt"], s["xt_scale"], "rows").t()
        return {"dx": dx.to(dtype), "dw": dw.to(dtype), "dbias": g.sum(0).to(dtype)}
    if s["op"] == "clip":
        norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
        factor = (s["max_norm"] / norm).clamp(max=1.0)
        return {"norm": norm.float(), "grads": [(g.double() * factor).to(g.dtype) for g in s["grads"]]}
    dtype = _DTYPES[s["dtype"]]
    h, m = s["h"].float(), s["m"]
    weight = s["weight"].float()
    if s["op"] == "norm":
        n, stats = h, []
        if s["post"]:
            stats = [_stats(h, s["norm"])]
            n = (h - stats[0][0][:, None]) * stats[0][1][:, None] * s["post_weight"].float()
        if s["gate"] is not None:
            n = n * _gate_rows(s, m)[0]
        # the next norm reads the sum as it is kept
        r = (s["scale"] * s["x"].float() + n).to(dtype)
        stats.insert(0, _stats(r.float(), s["norm"]))
        y = (r.float() - stats[0][0][:, None]) * stats[0][1][:, None] * weight + s["bias"].float()
        if s["out"] == "fp8":
            return {"r": r, "y": _decode(*_encode(y, "rows", "e4m3"), "rows").to(torch.bfloat16)}
        return {"r": r, "y": y.to(dtype), "stats": torch.cat(stats)}
    dy, stats = s["dy"].float(), s["stats"]
    dr, rh = _norm_gradient(dy, s["r"].float(), weight, stats[:2], s["norm"])
    dr = dr + s["dr"].float()
    out = {"dx": s["scale"] * dr, "dweight": (dy * rh).sum(0), "dbias": dy.sum(0)}
    dn = dr
    if s["gate"] is not None:
        gate, each = _gate_rows(s, m)
        n = h
        if s["post"]:
            n = (h - stats[2][:, None]) * stats[3][:, None] * s["post_weight"].float()
        out["dgate"] = (dr * n).reshape(-1, each, n.shape[1]).sum(1).reshape(s["gate"].shape)
        dn = dr * gate
    if s["post"]:
        dh, hh = _norm_gradient(dn, h, s["post_weight"].float(), stats[2:], s["norm"])
        out["dpost_weight"] = (dn * hh).sum(0)
        dn = dh
    out["dh"] = dn
    return {k: v.to(dtype) for k, v in out.items()}


def _kernels(s):
    import int8_convolution_forward_amd as ci8

    if s["op"] == "quantize":
        r = ci8.quantize_fp8(s["x"], block=s["block"], transposed=s["transposed"], dtype=_FORMATS[s["format"]])
        out = {"x": ci8.dequantize_fp8(r[0], r[1], dtype=torch.bfloat16)}
        if s["transposed"]:
            out["xt"] = ci8.dequantize_fp8(r[2], r[3], dtype=torch.bfloat16)
        return out
    if s["op"] == "linear":
        dtype = _DTYPES[s["out"]]
        z = torch.empty(s["m"], s["n"], dtype=dtype, device="cuda") if s["keep"] else None
        y = ci8.linear_fp8(s["x"], s["w"], s["x_scale"], s["w_scale"], bias=s["bias"], activation=s["act"],
                           residual=s.get("res"), out_dtype=dtype, preact=z)
        return {"y": y, "z": z} if s["keep"] else {"y": y}
    if s["op"] == "linear_backward":
        dx, dw, db = ci8.linear_fp8_backward(s["dy"], s["xt"], s["xt_scale"], s["wt"], s["wt_scale"], preact=s["z"],
                                             activation=s["act"], g_dtype=_FORMATS[s["format"]])
        return {"dx": dx, "dw": dw, "dbias": db}
    if s["op"] == "clip":
        norm = ci8.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
        return {"norm": norm, "grads": s["out"] if s["out"] is not None else s["grads"]}
    given = dict(weight=s["weight"], gate=s["gate"], post_weight=s["post_weight"], scale=s["scale"], norm=s["norm"])
    if s["op"] == "norm":
        if s["out"] == "fp8":
            r, q, scale = ci8.residual_norm_fp8(s["x"], s["h"], bias=s["bias"], eps=EPS, **given)
            return {"r": r, "y": ci8.dequantize_fp8(q, scale, dtype=torch.bfloat16)}
        r, y, stats = ci8.residual_norm(s["x"], s["h"], bias=s["bias"], eps=EPS, **given)
        return {"r": r, "y": y, "stats": stats}
    grads = ci8.residual_norm_backward(s["dr"], s["dy"], s["r"], s["h"], s["stats"], **given)
    names = ("dx", "dh", "dweight", "dbias", "dgate", "dpost_weight")
    out = {k: v for k, v in zip(names, grads) if v is not None}
    order = ("dx", "dweight", "dbias", "dgate", "dpost_weight", "dh")
    return {k: out[k] for k in order if k in out}


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    e = {"bf16": 2, "fp16": 2, "fp32": 4}[case.get("dtype", case.get("out"))]
    if case["op"] == "clip":
        count = sum(math.prod(shape) for shape in _shapes(case["tensors"], case["width"]))
        return {"bytes": count * e * (2 if case["clips"] else 1) + 4, "flops": count * (3 if case["clips"] else 2)}
    m = case["m"]
    if case["op"] == "quantize":
        k, copies = case["k"], 2 if case["transposed"] else 1
        # each copy is written in one byte and a scale, read again, and handed back in two
        return {"bytes": m * k * (e + copies * 4), "flops": 3 * m * k * copies}
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        kb = -(-k // BLOCK)
        moved = (m + n) * k + m * kb + -(-n // BLOCK) * kb + n * e
        return {"bytes": moved + m * n * e * (1 + bool(case["residual"]) + bool(case["keep"])), "flops": 2 * m * n * k}
    if case["op"] == "linear_backward":
        n, k = case["n"], case["k"]
        moved = m * n * (1 if case["act"] == "none" else 2) * e + (m + n) * k + -(-m // BLOCK) * k
        return {"bytes": moved + (m * k + n * k + n) * e, "flops": 4 * m * n * k}
    d = case["d"]
    gates = 0 if case["gate"] == "none" else 1 if case["gate"] == "vector" else _sequences(m)
    params = (2 + bool(case["post"]) + gates) * d * e
    stats = (2 + 2 * bool(case["post"])) * m * 4
    if case["op"] == "norm":
        # x, h and r; y in its own type, or written in one byte, read again and handed back in two
        out = 4 if case["out"] == "fp8" else e
        return {"bytes": m * d * (3 * e + out) + params + (0 if case["out"] == "fp8" else stats), "flops": 20 * m * d}
    # dr, dy and r, h where its values are needed; dx and dh
    reads = 3 + (case["post"] or case["gate"] != "none")
    return {"bytes": m * d * e * (reads + 2) + 2 * params + stats, "flops": 30 * m * d}


def _exact_quantised(x, block, form):
    """The numbers that x's quantised values stand for, in float64 by arithmetic alone."""
    bits, least, top = _MANTISSA[form]
    largest = (2 - 2.0 ** (1 - bits)) * 2.0 ** top if form == "e4m3" else (2 - 2.0 ** -bits) * 2.0 ** top
    b = _blocks(x, block)
    peak = b.abs().amax((1, 3), keepdim=True)
    e = torch.ceil(torch.log2(peak / largest)).clamp(-127, 127)
    e = torch.where(peak * torch.exp2(1 - e) <= largest, e - 1, e)  # where the logarithm rounded up
    e = torch.where(peak * torch.exp2(-e) > largest, e + 1, e).clamp_min(-127)
    e = torch.where(peak > 0, e, torch.full_like(e, -127.0))
    v = b * torch.exp2(-e)
    power = torch.floor(torch.log2(v.abs())).clamp_min(least)
    power = torch.where(torch.exp2(power) > v.abs(), power - 1, power).clamp_min(least)
    step = torch.exp2(power - bits)
    v = torch.round(v / step) * step * torch.exp2(e)
    return v.reshape(v.shape[0] * v.shape[1], -1)[:x.shape[0], :x.shape[1]]


def _exact_values(q, scale, tiles):
    """q's values times its blocks' scales, in float64."""
    m, k = q.shape
    rows = torch.arange(m, device=q.device) // (BLOCK if tiles else 1)
    cols = torch.arange(k, device=q.device) // BLOCK
    power = torch.exp2(scale.view(torch.uint8).double() - 127)
    return q.to(torch.float32).double() * power[rows][:, cols]


def _exact_act(z, act):
    """(act(z), act'(z)) in float64, from the definitions with the Gaussian
    distribution function written through erfc."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / 2 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        # 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
        u = (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        p = 1 / (1 + torch.exp(-2 * u))
        return z * p, p + z * p * (1 - p) * 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * z ** 2)
    p = 1 / (1 + torch.exp(-z))
    return z * p, p + z * p * (1 - p)


def _exact_normed(x, norm):
    """(normed x, mean, 1 / deviation) in float64."""
    if norm == "layer":
        var, mean = torch.var_mean(x, 1, correction=0)
    else:
        var, mean = torch.linalg.vecdot(x, x, dim=1) / x.shape[1], torch.zeros(x.shape[0], dtype=x.dtype, device=x.device)
    rstd = 1 / torch.sqrt(var + EPS)
    return (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), mean, rstd


def exact(case, seed):
    """The definitions above, written out in float64."""
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["x"].double()
        out = {"x": _exact_quantised(x, case["block"], case["format"])}
        if case["transposed"]:
            out["xt"] = _exact_quantised(x.T.contiguous(), case["block"], case["format"])
        return out
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        factor = min(1.0, s["max_norm"] / norm)
        return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [g.double() * factor for g in s["grads"]]}
    if case["op"] == "linear":
        x, w = _exact_values(s["x"], s["x_scale"], False), _exact_values(s["w"], s["w_scale"], True)
        z = torch.matmul(x, w.T) + s["bias"].double()
        y = _exact_act(z, case["act"])[0]
        if case["residual"]:
            y = y + s["res"].double()
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    if case["op"] == "linear_backward":
        g = s["dy"].double()
        if case["act"] != "none":
            g = g * _exact_act(s["z"].double(), case["act"])[1]
        dx = torch.matmul(_exact_quantised(g, "rows", case["format"]), _exact_values(s["wt"], s["wt_scale"], True).T)
        dw = torch.matmul(_exact_quantised(g.T.contiguous(), "rows", case["format"]),
                          _exact_values(s["xt"], s["xt_scale"], False).T)
        return {"dx": dx, "dw": dw, "dbias": g.sum(0)}
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    m, d = case["m"], case["d"]
    h, weight = wide["h"], wide["weight"]
    gates = wide["gate"].reshape(-1, d) if "gate" in wide else None
    if case["op"] == "norm":
        n, left = h, []
        if case["post"]:
            hh, mean, rstd = _exact_normed(h, case["norm"])
            n, left = hh * wide["post_weight"], [mean, rstd]
        if gates is not None:
            n = (n.reshape(gates.shape[0], -1, d) * gates.unsqueeze(1)).reshape(m, d)
        r = s["scale"] * wide["x"] + n
        # the norm is that of the sum as it is kept, rounded to the type of x
        rh, mean, rstd = _exact_normed(r.to(s["x"].dtype).double(), case["norm"])
        y = rh * weight + wide["bias"]
        if case["out"] == "fp8":
            return {"r": r, "y": _exact_quantised(y, "rows", "e4m3")}
        return {"r": r, "y": y, "stats": torch.stack([mean, rstd] + left)}
    stats, dy = wide["stats"].unsqueeze(2), wide["dy"]
    rh = (wide["r"] - stats[0]) * stats[1]
    c = dy * weight
    inner = c - rh * torch.mean(c * rh, 1, keepdim=True)
    dr = wide["dr"] + stats[1] * (inner - c.mean(1, keepdim=True) if case["norm"] == "layer" else inner)
    out = {"dx": s["scale"] * dr, "dweight": torch.sum(dy * rh, 0), "dbias": torch.sum(dy, 0)}
    hh = (h - stats[2]) * stats[3] if case["post"] else h
    dn = dr
    if gates is not None:
        n = hh * wide["post_weight"] if case["post"] else hh
        out["dgate"] = torch.sum((dr * n).reshape(gates.shape[0], -1, d), 1).reshape(wide["gate"].shape)
        dn = (dr.reshape(gates.shape[0], -1, d) * gates.unsqueeze(1)).reshape(m, d)
    if case["post"]:
        out["dpost_weight"] = torch.sum(dn * hh, 0)
        c = dn * wide["post_weight"]
        inner = c - hh * torch.mean(c * hh, 1, keepdim=True)
        dn = stats[3] * (inner - c.mean(1, keepdim=True) if case["norm"] == "layer" else inner)
    out["dh"] = dn
    return out
