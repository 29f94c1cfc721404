"""Low-rank adapters and 8-bit activation checkpoints: what is timed, the plain forms and the exact values.

The operators, as a user reaches them in ``split_gemm_gb300``:

  adapter_fwd      out = act(y + b_e h), h = scale_e a_e x: beside the shared projection's y, each row of x with
                   the adapter e that its entry of an index names (or none)
  adapter_bwd      its gradients: dx = dx0 + a_e^T dh with dh = scale_e b_e^T dy, and da, db summed over the rows of
                   each adapter; x in 16 bits or as an 8-bit checkpoint
  mxint8_quantize  8-bit integers in blocks of 32 with a shared power-of-two scale (MXINT8 of the OCP Microscaling
                   Formats specification), and mxint8_dequantize
  mxint8_layer_norm_bwd  the norm's gradient with x as such a checkpoint

``run`` computes them in elementary torch operations where ``own`` is false and through the package where it is
true.  A checkpoint of [rows, cols] is ``data`` int8 [rows, 32*ceil(cols/32)], zero past cols, and ``scales`` uint8
[rows, ceil(cols/32)]: element q of a block with scale byte s stands for q * 2^(s - 127 - 6); 255 marks NaN.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "int8": 33 / 32}
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
        # one token of one request, its adapter one of a pool of 64: the call's latency is all there is
        {"name": "adapter_one_token", "op": "adapter", "rows": 1, "cols": 4096, "outs": 4096, "rank": 16, "adapters": 64, "mix": "each",
         "none": False, "y": "bf16", "out": "bf16", "relu": False},
        # 64 requests decoded together, 32 adapters among them
        {"name": "adapter_decode", "op": "adapter", "rows": 64, "cols": 4096, "outs": 4096, "rank": 16, "adapters": 32, "mix": "each",
         "none": False, "y": "bf16", "out": "bf16", "relu": False},
        # a ragged batch of a few prompts, no extent a multiple of a vector's, the projection's result still in 32 bits
        {"name": "adapter_ragged", "op": "adapter", "rows": 777, "cols": 1001, "outs": 2001, "rank": 20, "adapters": 5, "mix": "runs",
         "none": True, "y": "f32", "out": "bf16", "relu": True},
        # prompts of 16 requests in one batch
        {"name": "adapter_prompts", "op": "adapter", "rows": 8192, "cols": 4096, "outs": 4096, "rank": 64, "adapters": 16, "mix": "runs",
         "none": True, "y": "bf16", "out": "bf16", "relu": False},
        # beside a 256 -> 1024 pointwise convolution of 16 x 28 x 28 pixels, one adapter, ReLU after it
        {"name": "adapter_28x28", "op": "adapter", "rows": 12544, "cols": 256, "outs": 1024, "rank": 16, "adapters": 1, "mix": "runs",
         "none": False, "y": "f32", "out": "bf16", "relu": True},
        # training three adapters on a small ragged batch, rows of each anywhere in it
        {"name": "adapter_grad_odd", "op": "adapter_grad", "rows": 785, "cols": 1001, "outs": 777, "rank": 8, "adapters": 3, "mix": "mixed",
         "none": True, "x": "bf16", "dx": "f32"},
        # the gradients beside the pointwise convolution, x kept in 8 bits
        {"name": "adapter_grad_28x28", "op": "adapter_grad", "rows": 12544, "cols": 256, "outs": 1024, "rank": 16, "adapters": 1,
         "mix": "runs", "none": False, "x": "int8", "dx": "bf16"},
        # four tasks trained together on long sequences beside one frozen layer, x kept in 8 bits
        {"name": "adapter_grad_large", "op": "adapter_grad", "rows": 16384, "cols": 4096, "outs": 4096, "rank": 64, "adapters": 4,
         "mix": "runs", "none": False, "x": "int8", "dx": "bf16"},
        # a small odd layer's activations into a checkpoint and back
        {"name": "checkpoint_odd", "op": "checkpoint", "rows": 333, "cols": 1001, "x": "f32"},
        # a long batch of a wide layer
        {"name": "checkpoint_large", "op": "checkpoint", "rows": 32768, "cols": 4096, "x": "bf16"},
        # the norm's gradient from a checkpoint: a ragged batch, channels no multiple of a vector
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 785, "cols": 1001, "dy": "f32"},
        # and at full length
        {"name": "norm_grad_large", "op": "norm_grad", "rows": 32768, "cols": 4096, "dy": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapter", "adapter", "adapter_grad", "adapter_grad", "checkpoint", "norm_grad"])
    if op in ("checkpoint", "norm_grad"):
        cols = _log(rng, 16, 16384)
        rows = _log(rng, 1, min(401408, 32768 * 4096 // cols))
        t = rng.choice(["bf16", "f32"])
        if t == "f32":
            rows = max(1, rows // 2)
        return {"op": op, "rows": rows, "cols": cols, ("x" if op == "checkpoint" else "dy"): t}
    cols, outs, rank = _log(rng, 64, 8192), _log(rng, 64, 8192), _log(rng, 4, 128)
    if rng.random() < 0.6:  # most layers' extents are whole vectors
        cols, outs, rank = cols // 8 * 8, outs // 8 * 8, max(1, rank // 8) * 8
    adapters = _log(rng, 1, min(128, max(1, 16 * 64 * 8192 // (rank * (cols + outs)))))
    rows = _log(rng, 1, min(16384, 8192 * 8192 // (cols + outs)))
    case = {"op": op, "rows": rows, "cols": cols, "outs": outs, "rank": rank, "adapters": adapters,
            "mix": rng.choice(["each", "runs", "mixed"]), "none": rng.random() < 0.5}
    if op == "adapter":
        case.update(y=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]), relu=rng.random() < 0.3)
    else:
        case.update(x=rng.choice(["bf16", "int8"]), dx=rng.choice(["bf16", "bf16", "f32"]))
    return case


# ----------------------------------------------------------------------------- inputs
def _activations(gen, rows, cols, dtype):
    """What a layer's output looks like: a spread and an offset of its own for each channel, a few channels far wider."""
    spread = torch.exp(0.5 * torch.randn(cols, device="cuda", generator=gen))
    wide = torch.rand(cols, device="cuda", generator=gen) < 0.01
    spread = torch.where(wide, 8 * spread, spread)
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    return x.mul_(spread).add_(0.3 * torch.randn(cols, device="cuda", generator=gen)).to(dtype)


def _index(gen, case):
    """Which adapter each row has: "each": neighbouring rows are different requests; "runs": a request's rows follow one another,
    their number anything; "mixed": any row, any adapter.  With "none" some rows have none (-1)."""
    rows, adapters = case["rows"], case["adapters"]
    ids = torch.randperm(adapters, device="cuda", generator=gen)
    if case["mix"] == "runs":
        if case["none"]:
            ids = torch.cat((ids[: adapters // 2], ids.new_tensor([-1]), ids[adapters // 2:]))
        n = min(len(ids), rows)
        cuts = torch.sort(1 + torch.randperm(rows - 1, device="cuda", generator=gen)[: n - 1]).values if n > 1 else ids[:0]
        return ids[torch.bucketize(torch.arange(rows, device="cuda"), cuts, right=True)].int()
    if case["mix"] == "each":
        index = ids.repeat(-(-rows // adapters))[:rows]
    else:
        index = torch.cat((ids, torch.randint(adapters, (rows,), device="cuda", generator=gen)))[:rows]
        index = index[torch.randperm(rows, device="cuda", generator=gen)]
    if case["none"]:
        index = torch.where(torch.rand(rows, device="cuda", generator=gen) < 0.1, -1, index)
    return index.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op, rows, cols = case["op"], case["rows"], case["cols"]
    if op == "checkpoint":
        s["x"] = _activations(gen, rows, cols, DTYPES[case["x"]])
    elif op == "norm_grad":
        x = _activations(gen, rows, cols, torch.float32)
        s["weight"] = 1 + 0.2 * torch.randn(cols, device="cuda", generator=gen)
        s["dy"] = (0.01 * torch.randn(rows, cols, device="cuda", generator=gen)).to(DTYPES[case["dy"]])
        s["mean"] = x.mean(1)
        s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
        s["x"] = _plain_quantize(x)
    else:
        outs, rank, adapters = case["outs"], case["rank"], case["adapters"]
        s["index"] = _index(gen, case)
        if own:  # made once for a batch and used beside every layer
            s["plan"] = _sg().adapter_plan(s["index"], adapters)
        s["a"] = (torch.randn(adapters, rank, cols, device="cuda", generator=gen) / math.sqrt(cols)).bfloat16()
        s["b"] = (torch.randn(adapters, outs, rank, device="cuda", generator=gen) * 0.5 / math.sqrt(rank)).bfloat16()
        s["scale"] = 0.5 + torch.rand(adapters, device="cuda", generator=gen)
        x = _activations(gen, rows, cols, torch.bfloat16)
        if op == "adapter":
            s["x"] = x
            s["y"] = torch.randn(rows, outs, device="cuda", generator=gen).to(DTYPES[case["y"]])
        else:
            s["dy"] = (0.01 * torch.randn(rows, outs, device="cuda", generator=gen)).bfloat16()
            s["dx0"] = (0.01 * torch.randn(rows, cols, device="cuda", generator=gen)).to(DTYPES[case["dx"]])
            s["h"] = torch.zeros(rows, rank, device="cuda")
            for e in range(adapters):
                here = (s["index"] == e).nonzero()[:, 0]
                s["h"][here] = s["scale"][e] * (x[here].float() @ s["a"][e].float().T)
            s["x"] = _plain_quantize(x) if case["x"] == "int8" else x
    return s


# ----------------------------------------------------------------------------- the plain forms
def _power(e):
    """2^e for whole e from -127 to 127, exactly (torch.ldexp and pow may be off by a bit, which would move ties)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _plain_quantize(x):
    rows, cols = x.shape
    blocks = -(-cols // 32)
    v = torch.nn.functional.pad(x.float(), (0, 32 * blocks - cols)).view(rows, blocks, 32)
    e = (v.abs().amax(2).view(torch.int32) >> 23) - 127  # floor(log2(the largest))
    bad = ~torch.isfinite(v).all(2)
    e = torch.where(bad, 0, e)
    q = torch.round((v * _power(-e).unsqueeze(2)) * 64).clamp(min=-127, max=127)  # ties to even
    q = torch.where(bad.unsqueeze(2), torch.zeros_like(q), q).to(torch.int8)
    return {"data": q.view(rows, 32 * blocks), "scales": torch.where(bad, 255, e + 127).to(torch.uint8), "rows": rows, "cols": cols}


def _plain_values(q):
    rows, cols = q["rows"], q["cols"]
    f = torch.where(q["scales"] == 255, float("nan"), _power(q["scales"].int() - 127))
    return ((q["data"].view(rows, -1, 32).float() / 64) * f.unsqueeze(2)).view(rows, -1)[:, :cols]


def _plain_masked(h, s):
    """[rows, adapters*rank] products with every adapter, those of a row's own scaled and the others zero."""
    case = s["case"]
    mine = s["index"][:, None] == torch.arange(case["adapters"], device="cuda")
    h = h.view(case["rows"], case["adapters"], case["rank"]) * s["scale"][:, None]
    return torch.where(mine.unsqueeze(2), h, torch.zeros_like(h)).view(case["rows"], -1)


def _plain_own_part(h, s):
    return h.view(s["case"]["rows"], s["case"]["adapters"], -1).sum(1)  # zeros but for the row's own


def _plain_adapter(s):
    case = s["case"]
    a = s["a"].float().flatten(0, 1)                        # [adapters*rank, cols]
    b = s["b"].float().permute(0, 2, 1).flatten(0, 1)       # [adapters*rank, outs]
    h = _plain_masked(s["x"].float() @ a.T, s)
    out = s["y"].float() + h @ b
    if case["relu"]:
        out = torch.clamp(out, min=0)
    return {"out": out.to(DTYPES[case["out"]]), "h": _plain_own_part(h, s)}


def _plain_adapter_grad(s):
    case = s["case"]
    a = s["a"].float().flatten(0, 1)
    b = s["b"].float().permute(0, 2, 1).flatten(0, 1)
    x = _plain_values(s["x"]) if case["x"] == "int8" else s["x"].float()
    dy = s["dy"].float()
    dh = _plain_masked(dy @ b.T, s)
    dx = s["dx0"].float() + dh @ a
    mine = s["index"][:, None] == torch.arange(case["adapters"], device="cuda")
    h = torch.where(mine.unsqueeze(2), s["h"].unsqueeze(1), torch.zeros((), device="cuda")).flatten(1)
    return {"dx": dx.to(DTYPES[case["dx"]]), "da": (dh.T @ x).view(s["a"].shape),
            "db": (dy.T @ h).view(case["outs"], case["adapters"], case["rank"]).permute(1, 0, 2).contiguous()}


def _plain_norm_grad(s):
    x, dy = _plain_values(s["x"]), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _plain(s):
    op = s["case"]["op"]
    if op == "adapter":
        return _plain_adapter(s)
    if op == "adapter_grad":
        return _plain_adapter_grad(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    return {"x": _plain_values(_plain_quantize(s["x"])).to(s["x"].dtype)}


# ----------------------------------------------------------------------------- through the package
def _own(s):
    sg, case = _sg(), s["case"]
    op = case["op"]
    if op == "checkpoint":
        return {"x": sg.mxint8_dequantize(sg.mxint8_quantize(s["x"]), out_dtype=s["x"].dtype)}
    if op == "norm_grad":
        dx, dw, db = sg.mxint8_layer_norm_bwd(s["dy"], sg.Mxint8(**s["x"]), s["mean"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    plan = s["plan"] if "plan" in s else sg.adapter_plan(s["index"], case["adapters"])
    if op == "adapter":
        out, h = sg.adapter_fwd(s["y"], s["x"], s["a"], s["b"], plan, s["scale"], relu=case["relu"], out_dtype=DTYPES[case["out"]])
        return {"out": out, "h": h}
    x = sg.Mxint8(**s["x"]) if case["x"] == "int8" else s["x"]
    dx, da, db = sg.adapter_bwd(s["dy"], x, s["h"], s["a"], s["b"], plan, s["scale"], dx=s["dx0"])
    return {"dx": dx, "da": da, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- work
def work(case):
    op, rows, cols = case["op"], case["rows"], case["cols"]
    e = rows * cols
    if op == "checkpoint":  # the checkpoint is written and read back
        return {"bytes": e * (2 * SIZE[case["x"]] + 2 * SIZE["int8"]), "flops": 6 * e}
    if op == "norm_grad":
        return {"bytes": e * (2 * SIZE[case["dy"]] + SIZE["int8"]) + 12 * cols + 8 * rows, "flops": 15 * e}
    outs, rank = case["outs"], case["rank"]
    weights = min(case["adapters"], rows) * rank * (cols + outs)  # of the adapters that rows have
    if op == "adapter":
        return {"bytes": 2 * e + 2 * weights + rows * outs * (SIZE[case["y"]] + SIZE[case["out"]]) + 4 * rows * (rank + 1),
                "flops": 2 * rows * rank * (cols + outs)}
    grads = case["adapters"] * rank * (cols + outs)
    return {"bytes": 2 * rows * outs + e * (SIZE[case["x"]] + 2 * SIZE[case["dx"]]) + 2 * weights + 4 * grads + 4 * rows * (rank + 1),
            "flops": 4 * rows * rank * (cols + outs)}


# ----------------------------------------------------------------------------- exact values, in 64 bits
def _exact_values(q):
    # a whole power of two is built in its bits, as exp2 need not be exact
    step = (q["scales"].long() - 127 - 6 + 1023 << 52).view(torch.float64)
    return (q["data"].double() * step.repeat_interleave(32, 1))[:, : q["cols"]]


def _exact_round_trip(x):
    x = x.double()
    rows, cols = x.shape
    v = torch.cat((x, x.new_zeros(rows, -cols % 32)), 1).view(rows, -1, 32)
    amax = v.abs().max(2, keepdim=True).values
    # frexp's mantissa lies in [1/2, 1); a step is a 64th of the power of two at or below the largest
    step = ((torch.frexp(amax).exponent.long() - 1).clamp(min=-127) - 6 + 1023 << 52).view(torch.float64)
    m = v.abs() / step
    low = m.floor()
    rest = m - low
    up = (rest > 0.5) | ((rest == 0.5) & (low % 2 == 1))
    out = torch.minimum(low + up.double(), torch.full_like(low, 127))
    return (torch.copysign(out, v) * step).view(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        return {"x": _exact_round_trip(s["x"])}
    if op == "norm_grad":
        n = case["cols"]
        dy, r = s["dy"].double(), s["rstd"].double()
        xc = _exact_values(s["x"]) - s["mean"].double()[:, None]
        g = dy * s["weight"].double()
        # by the chain through the mean and the deviation, not through the normalised value
        dot = (g * xc).sum(1) * r ** 3 / n
        dx = g * r[:, None] - (g.sum(1) * r / n)[:, None] - xc * dot[:, None]
        return {"dx": dx, "dweight": ((dy * xc) * r[:, None]).sum(0), "dbias": dy.sum(0)}
    a, b, scale = s["a"].double(), s["b"].double(), s["scale"].double()
    x = _exact_values(s["x"]) if case.get("x") == "int8" else s["x"].double()
    rows_of = [(s["index"] == e).nonzero()[:, 0] for e in range(case["adapters"])]
    if op == "adapter":
        out, h = s["y"].double(), x.new_zeros(case["rows"], case["rank"])
        for e, r in enumerate(rows_of):
            h[r] = torch.einsum("tc,rc->tr", x[r], a[e]) * scale[e]
            out[r] += torch.einsum("tr,kr->tk", h[r], b[e])
        return {"out": out.clamp_(min=0) if case["relu"] else out, "h": h}
    dy, h = s["dy"].double(), s["h"].double()
    dx, da, db = s["dx0"].double(), torch.zeros_like(a), torch.zeros_like(b)
    for e, r in enumerate(rows_of):
        dh = torch.einsum("tk,kr->tr", dy[r], b[e]) * scale[e]
        dx[r] += torch.einsum("tr,rc->tc", dh, a[e])
        da[e] = torch.einsum("tr,tc->rc", dh, x[r])
        db[e] = torch.einsum("tk,tr->kr", dy[r], h[r])
    return {"dx": dx, "da": da, "db": db}
