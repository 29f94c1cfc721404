"""Layer normalisation and microscaled 4-bit products: what is timed, the plain forms and the exact values.

The operators, as a user reaches them in ``split_gemm_gb300``:

  layer_norm_fwd     y = (x - mean) * rstd * weight + bias over the last dimension, with mean and rstd
  layer_norm_bwd     its gradient: dx, and dweight and dbias summed over all rows
  mxfp4_quantize     4-bit floating point (E2M1) in blocks of 32 with a shared power-of-two scale (E8M0):
                     of the rows, of the transpose, or of both in one pass; mxfp4_dequantize goes back
  mxfp4_matmul       y = relu(a b^T + bias) of two quantised operands
  layer_norm_mxfp4   the norm's output quantised without ever being written in 16 bits

``run`` computes them in elementary torch operations where ``own`` is false and through the package where
it is true.  A quantised matrix [rows, cols] is held as ``data`` [rows, 16*ceil(cols/32)] bytes (element 2j of
a row in the low half of byte j) and ``scales``, one byte per block of 32, in tiles of 128 rows x 4 blocks
(512 bytes; row r, block b at 16*(r%32) + 4*(r%128//32) + b%4; tiles row-major, padding zero).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5
_package = None


def _sg():
    global _package
    if _package is None:
        import split_gemm_gb300
        _package = split_gemm_gb300
    return _package


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a decoding step: the call's latency is all there is
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "x": "bf16", "y": "bf16"},
        # a long batch of tokens of a wide model
        {"name": "norm_large", "op": "norm", "rows": 32768, "cols": 4096, "x": "bf16", "y": "bf16"},
        # training on a ragged batch, channels no multiple of a vector
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 785, "cols": 1001, "x": "f32", "y": "f32"},
        # training at full length: the weight's gradient sums 32768 rows
        {"name": "norm_grad_large", "op": "norm_grad", "rows": 32768, "cols": 4096, "x": "bf16", "y": "bf16"},
        # weights or activations of an odd layer, quantised and read back
        {"name": "quantize_odd", "op": "quantize", "rows": 333, "cols": 1000, "form": "rows", "x": "bf16"},
        # a training step's activations: by rows for the product, transposed for the weight's gradient
        {"name": "quantize_both_large", "op": "quantize", "rows": 16384, "cols": 4096, "form": "both", "x": "bf16"},
        # one token through a wide layer: the weights' bytes are what counts
        {"name": "product_one_token", "op": "product", "m": 1, "n": 16384, "k": 4096, "y": "bf16", "epi": "none"},
        # odd extents everywhere, the last block partly filled
        {"name": "product_odd", "op": "product", "m": 777, "n": 1001, "k": 2000, "y": "bf16", "epi": "bias"},
        # the weight gradient of a 256 -> 1024 pointwise convolution over 16 x 28 x 28 pixels: few tiles, a long sum
        {"name": "product_weight_grad", "op": "product", "m": 1024, "n": 256, "k": 12544, "y": "f32", "epi": "none"},
        # a large layer at a long batch
        {"name": "product_large", "op": "product", "m": 8192, "n": 8192, "k": 8192, "y": "bf16", "epi": "none"},
        # a few requests decoded together: norm, quantisation and product of one layer
        {"name": "norm_product_decode", "op": "norm_product", "m": 8, "n": 4096, "k": 4096, "x": "bf16", "y": "bf16", "epi": "bias"},
        # channel norm and 256 -> 1024 pointwise convolution of 16 x 28 x 28 pixels, from the convolution's fp32 output
        {"name": "norm_product_28x28", "op": "norm_product", "m": 12544, "n": 1024, "k": 256, "x": "f32", "y": "bf16", "epi": "bias_relu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "product", "product", "norm_product"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 16, 16384)
        rows = _log(rng, 1, min(401408, 32768 * 4096 // cols))
        x = rng.choice(["bf16", "f32"])
        if x == "f32":
            rows = max(1, rows // 2)
        return {"op": op, "rows": rows, "cols": cols, "x": x, "y": x if op == "norm_grad" else rng.choice(["bf16", "f32"])}
    if op == "quantize":
        cols = _log(rng, 32, 16384)
        rows = _log(rng, 1, min(131072, 16384 * 4096 // cols))
        return {"op": op, "rows": rows, "cols": cols, "form": rng.choice(["rows", "columns", "both"]), "x": rng.choice(["bf16", "f32"])}
    n, k = _log(rng, 64, 16384), _log(rng, 64, 16384)
    m = _log(rng, 1, max(1, min(16384, 8192 ** 3 // (n * k))))
    case = {"op": op, "m": m, "n": n, "k": k, "y": rng.choice(["bf16", "bf16", "f32"]), "epi": rng.choice(["none", "bias", "bias_relu"])}
    if op == "norm_product":
        case["x"] = rng.choice(["bf16", "f32"])
    return case


# ----------------------------------------------------------------------------- inputs
def _activations(gen, rows, cols, dtype):
    """What a layer's output looks like: a spread and an offset of its own for each channel, a few channels far wider."""
    spread = torch.exp(0.5 * torch.randn(cols, device="cuda", generator=gen))
    wide = torch.rand(cols, device="cuda", generator=gen) < 0.01
    spread = torch.where(wide, 8 * spread, spread)
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    return x.mul_(spread).add_(0.3 * torch.randn(cols, device="cuda", generator=gen)).to(dtype)


def _params(gen, cols):
    return 1 + 0.2 * torch.randn(cols, device="cuda", generator=gen), 0.1 * torch.randn(cols, device="cuda", generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        s["x"] = _activations(gen, case["rows"], case["cols"], DTYPES[case["x"]])
        s["weight"], s["bias"] = _params(gen, case["cols"])
        if op == "norm_grad":
            s["dy"] = (0.01 * torch.randn(case["rows"], case["cols"], device="cuda", generator=gen)).to(DTYPES[case["y"]])
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
    elif op == "quantize":
        s["x"] = _activations(gen, case["rows"], case["cols"], DTYPES[case["x"]])
    else:
        m, n, k = case["m"], case["n"], case["k"]
        if op == "product":
            s["a"] = _plain_quantize(_activations(gen, m, k, torch.float32))
        else:
            s["x"] = _activations(gen, m, k, DTYPES[case["x"]])
            s["weight"], s["shift"] = _params(gen, k)
        s["b"] = _plain_quantize(torch.randn(n, k, device="cuda", generator=gen) / math.sqrt(k))
        s["bias"] = 0.1 * torch.randn(n, device="cuda", generator=gen) if case["epi"] != "none" else None
    return s


# ----------------------------------------------------------------------------- the plain forms
def _power(e):
    """2^e for whole e from -127 to 127, exactly (torch.ldexp and pow may be off by a bit, which would move ties)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _plain_norm(x, weight, bias):
    x = x.float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    return d * rstd * weight + bias, mean[:, 0], rstd[:, 0]


def _plain_norm_grad(dy, x, mean, rstd, weight):
    dy, xh = dy.float(), (x.float() - mean[:, None]) * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def _plain_codes(x):
    """(4-bit codes [rows, 32*blocks], scale bytes [rows, blocks]) of x in blocks of 32 along its rows."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    v = torch.nn.functional.pad(x.float(), (0, 32 * blocks - cols)).view(rows, blocks, 32)
    e = ((v.abs().amax(2).view(torch.int32) >> 23) - 129).clamp(min=-127)  # floor(log2(the largest)) - 2
    bad = ~torch.isfinite(v).all(2)
    v = v * _power(-e).unsqueeze(2)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)       # ties to the even mantissa
    code = torch.where(a <= 2, 2 * a, torch.where(a <= 4, a + 2, a / 2 + 4))  # 0 .5 1 1.5 2 3 4 6 -> 0 .. 7
    code = torch.where(bad.unsqueeze(2), torch.zeros_like(code), code).to(torch.uint8) + 8 * torch.signbit(v).to(torch.uint8)
    return code.view(rows, 32 * blocks), torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _plain_quantize(x):
    rows, cols = x.shape
    code, scale = _plain_codes(x)
    data = code[:, 0::2] | (code[:, 1::2] << 4)
    pr, pb = -rows % 128, -scale.shape[1] % 4
    t = torch.nn.functional.pad(scale, (0, pb, 0, pr))
    t = t.view((rows + pr) // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return {"data": data.contiguous(), "scales": t, "rows": rows, "cols": cols}


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _plain_values(q):
    """The values that a quantised matrix stands for."""
    rows, cols = q["rows"], q["cols"]
    table = torch.tensor(_E2M1, device="cuda")
    d = q["data"].long()
    v = torch.stack((table[d & 15], table[d >> 4]), 2).view(rows, -1, 32)
    tr, tb = -(-rows // 128), -(-v.shape[1] // 4)
    s = q["scales"].view(tr, tb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128 * tr, 4 * tb)[:rows, : v.shape[1]]
    f = torch.where(s == 255, float("nan"), _power(s.int() - 127))
    return (v * f.unsqueeze(2)).view(rows, -1)[:, :cols]


def _plain_product(case, a, b, bias):
    y = a @ b.T
    if bias is not None:
        y = y + bias
    if case["epi"] == "bias_relu":
        y = torch.clamp(y, min=0)
    return y.to(DTYPES[case["y"]])


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd = _plain_norm(s["x"], s["weight"], s["bias"])
        return {"y": y.to(DTYPES[case["y"]]), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dx, dw, db = _plain_norm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"dx": dx.to(s["x"].dtype), "dweight": dw, "dbias": db}
    if op == "quantize":
        out = {}
        if case["form"] != "columns":
            out["rows"] = _plain_values(_plain_quantize(s["x"])).to(torch.bfloat16)
        if case["form"] != "rows":
            out["columns"] = _plain_values(_plain_quantize(s["x"].T)).to(torch.bfloat16)
        return out
    if op == "norm_product":
        a = _plain_values(_plain_quantize(_plain_norm(s["x"], s["weight"], s["shift"])[0]))
    else:
        a = _plain_values(s["a"])
    return {"y": _plain_product(case, a, _plain_values(s["b"]), s["bias"])}


# ----------------------------------------------------------------------------- through the package
def _own(s):
    sg, case = _sg(), s["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd = sg.layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS, out_dtype=DTYPES[case["y"]])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dx, dw, db = sg.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "quantize":
        if case["form"] == "both":
            r, c = sg.mxfp4_quantize_both(s["x"])
            return {"rows": sg.mxfp4_dequantize(r), "columns": sg.mxfp4_dequantize(c)}
        q = sg.mxfp4_quantize(s["x"], transpose=case["form"] == "columns")
        return {case["form"]: sg.mxfp4_dequantize(q)}
    if op == "norm_product":
        a = sg.layer_norm_mxfp4(s["x"], s["weight"], s["shift"], EPS)
    else:
        a = sg.Mxfp4(**s["a"])
    return {"y": sg.mxfp4_matmul(a, sg.Mxfp4(**s["b"]), s["bias"], relu=case["epi"] == "bias_relu", out_dtype=DTYPES[case["y"]])}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- work
def _mx_bytes(rows, cols):
    return rows * (cols / 2 + -(-cols // 32))


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        e = case["rows"] * case["cols"]
        if op == "norm":
            return {"bytes": e * (SIZE[case["x"]] + SIZE[case["y"]]) + 8 * case["cols"] + 8 * case["rows"], "flops": 8 * e}
        return {"bytes": e * (2 * SIZE[case["x"]] + SIZE[case["y"]]) + 12 * case["cols"] + 8 * case["rows"], "flops": 14 * e}
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        # quantised bytes are written and read back, and the values written in 16 bits
        forms = {"rows": (1, 0), "columns": (0, 1), "both": (1, 1)}[case["form"]]
        each = forms[0] * _mx_bytes(r, c) + forms[1] * _mx_bytes(c, r)
        return {"bytes": r * c * SIZE[case["x"]] + 2 * each + sum(forms) * r * c * 2, "flops": 5 * r * c * sum(forms)}
    m, n, k = case["m"], case["n"], case["k"]
    a = _mx_bytes(m, k) if op == "product" else m * k * SIZE[case["x"]] + 8 * k
    return {"bytes": a + _mx_bytes(n, k) + m * n * SIZE[case["y"]] + (4 * n if case["epi"] != "none" else 0),
            "flops": 2 * m * n * k + (9 * m * k if op == "norm_product" else 0)}


# ----------------------------------------------------------------------------- exact values, in 64 bits
def _exact_norm(x, weight, bias):
    x = x.double()
    n = x.shape[1]
    mean = x.sum(1) / n
    var = (x * x).sum(1) / n - mean * mean
    rstd = 1 / torch.sqrt(var + EPS)
    return ((x - mean[:, None]) * rstd[:, None]) * weight.double() + bias.double(), mean, rstd


def _exact_round_trip(x):
    """x in blocks of 32 along its rows, each value replaced by the nearest of the sixteen that its block's scale allows."""
    x = x.double()
    rows, cols = x.shape
    v = torch.cat((x, x.new_zeros(rows, -cols % 32)), 1).view(rows, -1, 32)
    amax = v.abs().max(2, keepdim=True).values
    # frexp's mantissa lies in [1/2, 1); a whole power of two is built in its bits, as exp2 need not be exact
    s = ((torch.frexp(amax).exponent.long() - 3).clamp(min=-127) + 1023 << 52).view(torch.float64)
    m = v.abs() / s
    out = torch.zeros_like(m)
    # midpoints between neighbours; True where a tie goes up to the even one
    for mid, up, value in ((0.25, False, 0.5), (0.75, True, 1.0), (1.25, False, 1.5), (1.75, True, 2.0), (2.5, False, 3.0), (3.5, True, 4.0), (5.0, False, 6.0)):
        out = torch.where((m >= mid) if up else (m > mid), value, out)
    return (torch.copysign(out, v) * s).view(rows, -1)[:, :cols]


def _exact_values(q):
    rows, cols = q["rows"], q["cols"]
    codes = torch.empty(rows, 2 * q["data"].shape[1], device="cuda", dtype=torch.float64)
    for half in (0, 1):
        c = (q["data"] >> (4 * half)) & 15
        e, f = ((c >> 1) & 3).double(), (c & 1).double()
        mag = torch.where(e == 0, f / 2, (1 + f / 2) * torch.where(e == 3, 4.0, e))  # 2^(e-1): 1, 2, 4
        codes[:, half::2] = torch.where(c >= 8, -mag, mag)
    b = torch.arange(codes.shape[1] // 32, device="cuda")
    r = torch.arange(rows, device="cuda")[:, None]
    at = ((r // 128) * -(-len(b) // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    s = (q["scales"][at].long() - 127 + 1023 << 52).view(torch.float64)
    return (codes * s.repeat_interleave(32, 1))[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        y, mean, rstd = _exact_norm(s["x"], s["weight"], s["bias"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        n = case["cols"]
        dy, r = s["dy"].double(), s["rstd"].double()
        xc = s["x"].double() - s["mean"].double()[:, None]
        g = dy * s["weight"].double()
        # by the chain through the mean and the deviation, not through the normalised value
        dot = (g * xc).sum(1) * r ** 3 / n
        dx = g * r[:, None] - (g.sum(1) * r / n)[:, None] - xc * dot[:, None]
        return {"dx": dx, "dweight": ((dy * xc) * r[:, None]).sum(0), "dbias": dy.sum(0)}
    if op == "quantize":
        out = {}
        if case["form"] != "columns":
            out["rows"] = _exact_round_trip(s["x"])
        if case["form"] != "rows":
            out["columns"] = _exact_round_trip(s["x"].T)
        return out
    if op == "norm_product":
        a = _exact_round_trip(_exact_norm(s["x"], s["weight"], s["shift"])[0])
    else:
        a = _exact_values(s["a"])
    y = a.matmul(_exact_values(s["b"]).t())
    if s["bias"] is not None:
        y += s["bias"].double()
    return {"y": y.clamp_(min=0) if case["epi"] == "bias_relu" else y}
