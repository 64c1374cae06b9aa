"""The gradient operators, as they are measured: embedding, layer norm and 8-bit products.

The step takes each worker's gradient of every weight as a stack [Mw][R][C]. These operators
are what a transformer's training pass needs to make those stacks: the embedding lookup and its
gradient by sorted tokens, layer norm and its gradients, the quantisation to 8-bit floating
point with a scale for each block of 128, and the product of such operands (a linear layer's
output, its input's gradient, or its weight's gradient by worker).

``run`` computes an operator in elementary torch operations, or, where ``own`` is true, calls
the library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2,
         "i32": torch.int32, "i64": torch.int64}
SIZE = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}
# exponent p of the largest value 0.875 * 2^p of a format: 448 = 0.875 * 2^9, 57344 = 0.875 * 2^16
TOP = {"e4m3": 9, "e5m2": 16}


def listed():
    return [
        # one prompt's tokens, looked up in the fp32 weights that the step updates
        {"name": "embed 64 tokens", "op": "embed", "workers": 1, "tokens": 64, "vocab": 32000, "cols": 768,
         "ids": "i64", "table": "f32", "x": "bf16", "scale": 1.0, "pad": False},
        # the gradient of a whole embedding table, eight workers' batches, for the step
        {"name": "embed grad 8 workers", "op": "embed_grad", "workers": 8, "tokens": 4096, "vocab": 32000, "cols": 768,
         "ids": "i64", "x": "bf16", "grad": "f32", "scale": 1.0, "add": False, "pad": False},
        # a ragged batch with padding, odd sizes, scaled by sqrt(cols)
        {"name": "embed grad odd", "op": "embed_grad", "workers": 3, "tokens": 1501, "vocab": 5003, "cols": 515,
         "ids": "i32", "x": "f32", "grad": "bf16", "scale": 22.7, "add": False, "pad": True},
        # a few rows of an odd width: latency
        {"name": "norm odd", "op": "norm", "rows": 100, "cols": 769, "x": "f32", "bias": True},
        # one layer norm of a small transformer, eight workers' batches
        {"name": "norm grad 8 workers", "op": "norm_grad", "workers": 8, "rows": 1024, "cols": 768, "x": "bf16",
         "grad": "f32", "bias": False},
        # one layer norm of a large block
        {"name": "norm grad 4096", "op": "norm_grad", "workers": 16, "rows": 1024, "cols": 4096, "x": "f32",
         "grad": "f32", "bias": True},
        # output gradients in the wider-range format, both ways, odd sizes
        {"name": "quant odd", "op": "f8_quant", "batch": 3, "rows": 1000, "cols": 1111, "x": "f32", "f8": "e5m2",
         "way": "both"},
        # a large block's weights, for the output and for the input's gradient
        {"name": "quant weights", "op": "f8_quant", "batch": 1, "rows": 11008, "cols": 4096, "x": "f32", "f8": "e4m3",
         "way": "both"},
        # one token through a large layer
        {"name": "matmul one row", "op": "f8_matmul", "batch": 1, "m": 1, "n": 11008, "k": 4096, "a": "e4m3",
         "b": "e4m3", "out": "bf16", "shared": True},
        # a small transformer's fused projection, eight workers' tokens
        {"name": "matmul projection", "op": "f8_matmul", "batch": 1, "m": 8192, "n": 2304, "k": 768, "a": "e4m3",
         "b": "e4m3", "out": "bf16", "shared": True},
        # eight workers' gradients of a small weight, summed over each worker's tokens
        {"name": "matmul weight grad", "op": "f8_matmul", "batch": 8, "m": 768, "n": 2304, "k": 2000, "a": "e5m2",
         "b": "e4m3", "out": "f32", "shared": False},
        # a large block's up projection
        {"name": "matmul block", "op": "f8_matmul", "batch": 1, "m": 16384, "n": 11008, "k": 4096, "a": "e4m3",
         "b": "e4m3", "out": "bf16", "shared": True},
    ]


MOST_BYTES = 9e8
MOST_FLOPS = 6e11


def _spread(rng, low, high):
    """A whole number, spread over the logarithm of [low, high]; about half of them multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "norm", "norm_grad", "norm_grad", "f8_quant", "f8_quant",
                     "f8_matmul", "f8_matmul", "f8_matmul"])
    while True:
        x = rng.choice(["f32", "bf16"])
        grad = rng.choice(["f32", "f32", "bf16"])
        if op in ("embed", "embed_grad"):
            case = {"op": op, "workers": rng.choice([1, 2, 3, 8]), "tokens": _spread(rng, 1, 16384),
                    "vocab": _spread(rng, 100, 65536), "cols": _spread(rng, 32, 4096), "ids": rng.choice(["i32", "i64"]),
                    "x": x, "scale": rng.choice([1.0, 8.0, 27.7]), "pad": rng.random() < 0.5}
            case |= {"table": grad} if op == "embed" else {"grad": grad, "add": rng.random() < 0.3}
        elif op == "norm":
            case = {"op": op, "rows": _spread(rng, 1, 32768), "cols": _spread(rng, 32, 16384), "x": x,
                    "bias": rng.random() < 0.5}
        elif op == "norm_grad":
            case = {"op": op, "workers": rng.choice([1, 2, 3, 8]), "rows": _spread(rng, 1, 8192),
                    "cols": _spread(rng, 32, 16384), "x": x, "grad": grad, "bias": rng.random() < 0.5}
        elif op == "f8_quant":
            case = {"op": op, "batch": rng.choice([1, 1, 2, 5, 8]), "rows": _spread(rng, 1, 16384),
                    "cols": _spread(rng, 32, 16384), "x": x, "f8": rng.choice(["e4m3", "e5m2"]),
                    "way": rng.choice(["rows", "columns", "both", "both"])}
        else:
            batch = rng.choice([1, 1, 1, 3, 8])
            case = {"op": op, "batch": batch, "m": _spread(rng, 1, 16384), "n": _spread(rng, 64, 16384),
                    "k": _spread(rng, 64, 16384), "a": rng.choice(["e4m3", "e4m3", "e5m2"]),
                    "b": rng.choice(["e4m3", "e4m3", "e5m2"]), "out": grad, "shared": batch == 1 or rng.random() < 0.3}
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return case


def _up(n, to):
    return (n + to - 1) // to * to


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        tokens, c = case["workers"] * case["tokens"], case["cols"]
        some = case["workers"] * min(case["tokens"], case["vocab"])
        rows = tokens * (SIZE[case["ids"]] + c * SIZE[case["x"]])
        if op == "embed":
            return {"bytes": rows + min(tokens, case["vocab"]) * c * SIZE[case["table"]], "flops": tokens * c}
        grad = 2 * some * c if case["add"] else case["workers"] * case["vocab"] * c
        return {"bytes": rows + grad * SIZE[case["grad"]], "flops": 2 * tokens * c}
    if op == "norm":
        n, c = case["rows"], case["cols"]
        return {"bytes": 2 * n * c * SIZE[case["x"]] + 8 * n + 4 * c * (2 if case["bias"] else 1), "flops": 8 * n * c}
    if op == "norm_grad":
        n, c, sums = case["workers"] * case["rows"], case["cols"], 2 if case["bias"] else 1
        return {"bytes": 3 * n * c * SIZE[case["x"]] + 8 * n + 4 * c + sums * case["workers"] * c * SIZE[case["grad"]],
                "flops": 15 * n * c}
    if op == "f8_quant":
        b, r, c = case["batch"], case["rows"], case["cols"]
        out = (r * _up(c, 128) * 129 // 128 if case["way"] != "columns" else 0) + \
              (c * _up(r, 128) * 129 // 128 if case["way"] != "rows" else 0)
        return {"bytes": b * (r * c * SIZE[case["x"]] + out), "flops": 3 * b * r * c}
    b, m, n, k = case["batch"], case["m"], case["n"], case["k"]
    return {"bytes": (b * m + (1 if case["shared"] else b) * n) * k * 129 // 128 + b * m * n * SIZE[case["out"]],
            "flops": 2 * b * m * n * k}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _quant(x, f8):
    """x [..., k] in blocks of 128 along k: values times 2^-e, rounded to f8, and the bytes e + 127.
    e is the least exponent whose block fits the format (at least -127; 0 for a block of zeros).
    Rows are padded with zeros to a multiple of 128, scales with byte 127 to a multiple of 4."""
    k = x.shape[-1]
    kp, blocks = _up(k, 128), _up(_up(k, 128) // 128, 4)
    x = torch.nn.functional.pad(x.float(), (0, kp - k)).unflatten(-1, (kp // 128, 128))
    size = x.abs()
    top = torch.where(torch.isfinite(size), size, 0.0).amax(-1)
    m, p = torch.frexp(top)
    e = torch.where(top > 0, (p + (m > 0.875).int() - TOP[f8]).clamp(min=-127), 0)
    q = torch.ldexp(x, -e.unsqueeze(-1)).flatten(-2).to(TYPES[f8])
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, blocks - kp // 128), value=127)
    return q, s


def _tokens(case, g):
    """Token numbers whose frequency falls as one over their rank, as words' does."""
    u = torch.rand(case["workers"], case["tokens"], generator=g, device=DEV, dtype=torch.float64)
    ids = (float(case["vocab"] + 1) ** u).long().sub(1).clamp(0, case["vocab"] - 1)
    if case["pad"]:  # the tail of each worker's batch
        keep = torch.rand(case["workers"], 1, generator=g, device=DEV) * 0.3 + 0.7
        at = torch.arange(case["tokens"], device=DEV)
        ids = torch.where(at < (keep * case["tokens"]).ceil(), ids, -1)
    return ids.to(TYPES[case["ids"]])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    op, s = case["op"], {"case": case}
    if op in ("embed", "embed_grad"):
        w, t, v, c = case["workers"], case["tokens"], case["vocab"], case["cols"]
        s["ids"] = _tokens(case, g)
        if op == "embed":
            s["table"] = (normal(v, c) * 0.02).to(TYPES[case["table"]])
            s["y"] = torch.empty(w, t, c, dtype=TYPES[case["x"]], device=DEV)
        else:
            s["dy"] = (normal(w, t, c) * 1e-3).to(TYPES[case["x"]])
            s["grad"] = torch.empty(w, v, c, dtype=TYPES[case["grad"]], device=DEV)
            if case["add"]:  # what the output layer that shares the table has left there
                s["grad"].normal_(std=1e-3, generator=g)
    elif op in ("norm", "norm_grad"):
        n, c, x = case.get("workers", 1) * case["rows"], case["cols"], TYPES[case["x"]]
        s["x"] = (normal(n, c) * 2 + 0.5 * normal(c)).to(x)
        s["gamma"] = 1 + 0.1 * normal(c)
        s["eps"] = 1e-5
        if op == "norm":
            s["beta"] = 0.1 * normal(c) if case["bias"] else None
            s["y"] = torch.empty(n, c, dtype=x, device=DEV)
            s["mean"], s["rstd"] = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        else:
            s["dy"] = (normal(n, c) * 1e-3).to(x)
            s["mean"] = s["x"].float().mean(-1)
            s["rstd"] = torch.rsqrt(s["x"].float().var(-1, unbiased=False) + s["eps"])
            s["dx"] = torch.empty(n, c, dtype=x, device=DEV)
            s["dgamma"] = torch.empty(case["workers"], c, dtype=TYPES[case["grad"]], device=DEV)
            s["dbeta"] = torch.empty_like(s["dgamma"]) if case["bias"] else None
    elif op == "f8_quant":
        b, r, c, f8 = case["batch"], case["rows"], case["cols"], TYPES[case["f8"]]
        # rows of different sizes, as tokens' gradients are
        s["x"] = (normal(b, r, c) * torch.exp(2 * normal(b, r, 1)) * 0.02).to(TYPES[case["x"]])
        both = {"q": (b, r, c), "qt": (b, c, r)}
        for name in {"rows": ("q",), "columns": ("qt",), "both": ("q", "qt")}[case["way"]]:
            _, rows, cols = both[name]
            s[name] = torch.empty(b, rows, _up(cols, 128), dtype=f8, device=DEV)
            s[name + "_scale"] = torch.empty(b, rows, _up(_up(cols, 128) // 128, 4), dtype=torch.uint8, device=DEV)
    else:
        b, m, n, k = case["batch"], case["m"], case["n"], case["k"]
        s["a"], s["a_scale"] = _quant(normal(b, m, k) * torch.exp(normal(b, m, 1)), case["a"])
        s["b"], s["b_scale"] = _quant(normal(1 if case["shared"] else b, n, k) * 0.02, case["b"])
        s["out"] = torch.empty(b, m, n, dtype=TYPES[case["out"]], device=DEV)
    return s


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _call(s):
    import sign_muon_step_amd as sm

    case = s["case"]
    op = case["op"]
    if op == "embed":
        sm.signmuon_embedding(s["ids"], s["table"], case["scale"], s["y"])
        return s["y"]
    if op == "embed_grad":
        if "ws" not in s:
            s["ws"] = sm.bytes_tensor(sm.signmuon_embedding_workspace_bytes(
                case["workers"], case["tokens"], case["vocab"], case["cols"]), DEV)
        sm.signmuon_embedding_backward(s["ids"], s["dy"], case["scale"], s["grad"], s["ws"], accumulate=case["add"])
        return s["grad"]
    if op == "norm":
        sm.signmuon_layer_norm(s["x"], s["gamma"], s["beta"], s["eps"], s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_grad":
        if "ws" not in s:
            s["ws"] = sm.bytes_tensor(sm.signmuon_layer_norm_workspace_bytes(
                case["workers"], case["rows"], case["cols"]), DEV)
        sm.signmuon_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"],
                                        s["dbeta"], s["ws"], workers=case["workers"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "f8_quant":
        sm.signmuon_f8_quant(s["x"], s.get("q"), s.get("q_scale"), s.get("qt"), s.get("qt_scale"))
        return {k: s[k] for k in ("q", "q_scale", "qt", "qt_scale") if k in s}
    if "ws" not in s:
        s["ws"] = sm.bytes_tensor(sm.signmuon_f8_matmul_workspace_bytes(case["batch"], case["m"], case["n"], case["k"]),
                                  DEV)
    sm.signmuon_f8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], case["k"], s["out"], s["ws"])
    return s["out"]


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _values(q, s, k, dtype):
    """What 8-bit operands stand for: [..., k] of dtype."""
    e = s[..., : q.shape[-1] // 128].to(torch.int32) - 127
    x = q.to(dtype).unflatten(-1, (-1, 128))
    return torch.ldexp(x, e.unsqueeze(-1)).flatten(-2)[..., :k]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embed":
        ids = s["ids"].long()
        there = (ids >= 0) & (ids < case["vocab"])
        rows = s["table"][ids.clamp(0, case["vocab"] - 1)].float() * case["scale"]
        return torch.where(there.unsqueeze(-1), rows, 0.0).to(TYPES[case["x"]])
    if op == "embed_grad":
        v, w, c = case["vocab"], case["workers"], case["cols"]
        ids = s["ids"].long()
        there = (ids >= 0) & (ids < v)
        at = (ids + v * torch.arange(w, device=DEV).unsqueeze(1))[there]
        total = torch.zeros(w * v, c, device=DEV)
        total.index_add_(0, at, s["dy"][there].float())
        total = total.view(w, v, c) * case["scale"]
        if case["add"]:
            s["grad"].copy_(s["grad"].float() + total)
        else:
            s["grad"].copy_(total)
        return s["grad"]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(-1, keepdim=True)
        x = x - mean
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        y = x * rstd * s["gamma"]
        if s["beta"] is not None:
            y = y + s["beta"]
        return {"y": y.to(s["x"].dtype), "mean": mean.squeeze(-1), "rstd": rstd.squeeze(-1)}
    if op == "norm_grad":
        dy, w, c = s["dy"].float(), case["workers"], case["cols"]
        xhat = (s["x"].float() - s["mean"].unsqueeze(-1)) * s["rstd"].unsqueeze(-1)
        t = dy * s["gamma"]
        dx = (t - t.mean(-1, keepdim=True) - xhat * (t * xhat).mean(-1, keepdim=True)) * s["rstd"].unsqueeze(-1)
        grad = s["dgamma"].dtype
        return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).view(w, -1, c).sum(1).to(grad),
                "dbeta": dy.view(w, -1, c).sum(1).to(grad) if case["bias"] else None}
    if op == "f8_quant":
        out = {}
        if case["way"] != "columns":
            out["q"], out["q_scale"] = _quant(s["x"], case["f8"])
        if case["way"] != "rows":
            out["qt"], out["qt_scale"] = _quant(s["x"].transpose(1, 2), case["f8"])
        return out
    a = _values(s["a"], s["a_scale"], case["k"], torch.float32)
    b = _values(s["b"], s["b_scale"], case["k"], torch.float32).transpose(1, 2).contiguous()
    if case["shared"]:
        out = torch.matmul(a.flatten(0, 1), b[0]).view(case["batch"], case["m"], case["n"])
    else:
        out = torch.bmm(a, b)
    return out.to(TYPES[case["out"]])


def run(state):
    if own:
        return _call(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# In 64 bits
# ---------------------------------------------------------------------------
def _scaled(x, f8):
    """x over its blocks' scales, rounded to the format: to the nearest multiple of 2^(p - m), ties to
    even, p the value's exponent (at least the smallest normal one) and m the format's mantissa bits."""
    n, c = x.shape[-1], _up(x.shape[-1], 128)
    out = torch.zeros(*x.shape[:-1], c, dtype=torch.float64, device=x.device)
    out[..., :n] = x
    out = out.unflatten(-1, (-1, 128))
    largest = out.abs().amax(-1, keepdim=True)
    top = 0.875 * 2.0 ** TOP[f8]
    e = torch.ceil(torch.log2(largest / top))
    e = torch.where(largest > torch.exp2(e) * top, e + 1, e)
    e = torch.where(largest <= torch.exp2(e - 1) * top, e - 1, e)
    e = torch.where(largest > 0, e.clamp(min=-127), 0.0)
    out = (out / torch.exp2(e)).flatten(-2)
    mantissa, smallest = {"e4m3": (3, -6), "e5m2": (2, -14)}[f8]
    p = torch.floor(torch.log2(out.abs().clamp(min=2.0 ** -40))).clamp(min=smallest)
    step = torch.exp2(p - mantissa)
    return torch.round(out / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "embed":
        table = torch.cat([s["table"].to(f64), torch.zeros(1, case["cols"], dtype=f64, device=DEV)])
        ids = s["ids"].long()
        ids = torch.where((ids < 0) | (ids >= case["vocab"]), case["vocab"], ids)
        return table[ids] * case["scale"]
    if op == "embed_grad":
        out = []
        for w in range(case["workers"]):  # one worker after the other: the last row takes the padding
            ids = s["ids"][w].long()
            ids = torch.where((ids < 0) | (ids >= case["vocab"]), case["vocab"], ids)
            total = torch.zeros(case["vocab"] + 1, case["cols"], dtype=f64, device=DEV)
            total.index_put_((ids,), s["dy"][w].to(f64), accumulate=True)
            total = total[:-1] * case["scale"]
            out.append(total + s["grad"][w].to(f64) if case["add"] else total)
        return torch.stack(out)
    if op == "norm":
        x = s["x"].to(f64)
        var, mean = torch.var_mean(x, dim=-1, correction=0)
        rstd = 1 / torch.sqrt(var + s["eps"])
        y = (x - mean[:, None]) * rstd[:, None] * s["gamma"].to(f64)
        return {"y": y if s["beta"] is None else y + s["beta"].to(f64), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        w, c = case["workers"], case["cols"]
        dy, gamma, rstd = s["dy"].to(f64), s["gamma"].to(f64), s["rstd"].to(f64)[:, None]
        xhat = (s["x"].to(f64) - s["mean"].to(f64)[:, None]) * rstd
        t = dy * gamma
        # the projection of t off the vectors 1 and xhat, both of squared length c
        t = t - (t.sum(-1, keepdim=True) + xhat * (t * xhat).sum(-1, keepdim=True)) / c
        return {"dx": t * rstd, "dgamma": (dy * xhat).view(w, -1, c).sum(1),
                "dbeta": dy.view(w, -1, c).sum(1) if case["bias"] else None}
    if op == "f8_quant":
        out = {}
        if case["way"] != "columns":
            out |= {"q": _scaled(s["x"].to(f64), case["f8"]), "q_scale": None}
        if case["way"] != "rows":
            out |= {"qt": _scaled(s["x"].to(f64).transpose(1, 2), case["f8"]), "qt_scale": None}
        return out
    out = torch.empty(case["batch"], case["m"], case["n"], dtype=f64, device=DEV)
    for i in range(case["batch"]):
        j = 0 if case["shared"] else i
        a, b = s["a"][i].to(f64), s["b"][j].to(f64)
        a *= torch.exp2(s["a_scale"][i].to(f64) - 127).repeat_interleave(128, -1)[:, : a.shape[-1]]
        b *= torch.exp2(s["b_scale"][j].to(f64) - 127).repeat_interleave(128, -1)[:, : b.shape[-1]]
        out[i] = a @ b.t().contiguous()
    return out
