"""The operators around the training pass's two ends, as they are measured: the loss, the norm
with the residual stream, and gradient clipping.

The step takes each worker's gradient of every weight as a stack [Mw][R][C]. Between the norms
and 8-bit products that a pass has already and those stacks lie: root-mean-square norm with the
residual's addition, whose output may go straight to an 8-bit product; the softmax cross entropy
of an output layer, with the gradients of its input and of its weight; and the norm of each
worker's gradients over all weights, with clipping.

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
        # the score of one next token: latency and one pass over the output layer
        {"name": "loss 1 token", "op": "loss", "tokens": 1, "vocab": 32000, "cols": 768, "ids": "i64",
         "x": "bf16", "w": "bf16", "scale": 1.0, "pad": False},
        # evaluation of a small transformer on four sequences, padded
        {"name": "loss evaluation", "op": "loss", "tokens": 4096, "vocab": 50257, "cols": 768, "ids": "i64",
         "x": "bf16", "w": "bf16", "scale": 1.0, "pad": True},
        # a ragged batch of odd sizes with padding, all in fp32, its logits scaled
        {"name": "loss grad odd", "op": "loss_grad", "workers": 3, "tokens": 501, "vocab": 5003, "cols": 515,
         "ids": "i32", "x": "f32", "w": "f32", "grad": "f32", "scale": 0.75, "add": False, "pad": True},
        # the output layer of a small transformer, eight workers' batches, for the step
        {"name": "loss grad 8 workers", "op": "loss_grad", "workers": 8, "tokens": 1024, "vocab": 50257, "cols": 768,
         "ids": "i64", "x": "bf16", "w": "bf16", "grad": "f32", "scale": 1.0, "add": False, "pad": False},
        # the output layer above a large block
        {"name": "loss grad block", "op": "loss_grad", "workers": 1, "tokens": 8192, "vocab": 32000, "cols": 4096,
         "ids": "i64", "x": "bf16", "w": "bf16", "grad": "bf16", "scale": 1.0, "add": False, "pad": False},
        # one token between two layers of a large block: latency
        {"name": "norm 1 token", "op": "norm", "rows": 1, "cols": 4096, "x": "bf16", "residual": True, "y": True,
         "f8": "e4m3"},
        # eight workers' tokens on their way into an 8-bit projection
        {"name": "norm to 8 bits", "op": "norm", "rows": 8192, "cols": 768, "x": "bf16", "residual": True, "y": False,
         "f8": "e4m3"},
        # the same norm's gradients, with the residual stream's own
        {"name": "norm grad 8 workers", "op": "norm_grad", "workers": 8, "rows": 1024, "cols": 768, "x": "bf16",
         "grad": "f32", "residual": True},
        # odd sizes in fp32
        {"name": "norm grad odd", "op": "norm_grad", "workers": 3, "rows": 233, "cols": 5003, "x": "f32",
         "grad": "bf16", "residual": False},
        # one small matrix of four workers: latency
        {"name": "clip one matrix", "op": "clip", "workers": 4, "sizes": "256x256", "x": "f32", "most": 1.0},
        # every convolution and scale of a residual network's stage, odd sizes among them, in bf16
        {"name": "clip many", "op": "clip", "workers": 8, "x": "bf16", "most": 0.5,
         "sizes": "64x147 64x64*3 64x576*3 256x64*4 128x1152*4 512x128*4 256x2304*6 1024x256*6 1x64*10 1x256*8 1x1001 1001x2048"},
        # the matrices and norms of a large block, four workers
        {"name": "clip block", "op": "clip", "workers": 4, "sizes": "4096x4096*4 4096x11008 11008x4096 1x4096*2",
         "x": "f32", "most": 1.0},
    ]


MOST_BYTES = 8e9
MOST_FLOPS = 2e12


def _spread(rng, low, high):
    """A whole number, spread over the logarithm of [low, high]; about half of them multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["loss", "loss", "loss_grad", "loss_grad", "loss_grad", "norm", "norm", "norm_grad", "norm_grad",
                     "clip", "clip"])
    while True:
        x = rng.choice(["f32", "bf16", "bf16"])
        grad = rng.choice(["f32", "bf16"])
        if op in ("loss", "loss_grad"):
            case = {"op": op, "tokens": _spread(rng, 1, 8192), "vocab": _spread(rng, 100, 65536),
                    "cols": _spread(rng, 32, 8192), "ids": rng.choice(["i32", "i64"]), "x": x,
                    "w": rng.choice([x, x, "f32", "bf16"]), "scale": rng.choice([1.0, 1.0, 0.75, 0.0625]),
                    "pad": rng.random() < 0.5}
            if op == "loss_grad":
                case |= {"workers": rng.choice([1, 2, 3, 8]), "grad": grad, "add": rng.random() < 0.3}
                if case["workers"] * case["vocab"] * case["cols"] > 6e8:
                    continue
            if case.get("workers", 1) * case["tokens"] * case["vocab"] > 4.2e8:
                continue
        elif op == "norm":
            case = {"op": op, "rows": _spread(rng, 1, 32768), "cols": _spread(rng, 32, 16384), "x": x,
                    "residual": rng.random() < 0.7, "y": rng.random() < 0.5, "f8": rng.choice(["", "e4m3", "e4m3", "e5m2"])}
            if not case["y"] and not case["f8"]:
                continue
        elif op == "norm_grad":
            case = {"op": op, "workers": rng.choice([1, 2, 3, 8]), "rows": _spread(rng, 1, 8192),
                    "cols": _spread(rng, 32, 16384), "x": x, "grad": grad, "residual": rng.random() < 0.7}
        else:
            sizes = ["%dx%d*%d" % (_spread(rng, 1, 8192), _spread(rng, 1, 8192), rng.choice([1, 1, 2, 5, 20]))
                     for _ in range(rng.choice([1, 2, 3, 5, 8]))]
            case = {"op": op, "workers": rng.choice([1, 2, 3, 8]), "sizes": " ".join(sizes), "x": x,
                    "most": rng.choice([0.25, 1.0, 1e9])}
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return case


def _up(n, to):
    return (n + to - 1) // to * to


def _counts(sizes):
    """The number of entries of each tensor: "64x147 64x64*3" is one of 64 x 147 and three of 64 x 64."""
    out = []
    for part in sizes.split():
        shape, _, times = part.partition("*")
        rows, _, cols = shape.partition("x")
        out += [int(rows) * int(cols)] * int(times or 1)
    return out


def work(case):
    op = case["op"]
    if op in ("loss", "loss_grad"):
        t, v, c = case.get("workers", 1) * case["tokens"], case["vocab"], case["cols"]
        read = t * c * SIZE[case["x"]] + v * c * SIZE[case["w"]] + t * SIZE[case["ids"]] + 8 * t
        if op == "loss":
            return {"bytes": read, "flops": 2 * t * v * c}
        grad = t * c * SIZE[case["x"]] + case["workers"] * v * c * SIZE[case["grad"]] * (2 if case["add"] else 1)
        return {"bytes": read + grad + 4 * t, "flops": 6 * t * v * c}
    if op == "norm":
        n, c, e = case["rows"], case["cols"], SIZE[case["x"]]
        each = e * ((3 if case["residual"] else 1) + (1 if case["y"] else 0))
        return {"bytes": n * (c * each + (_up(c, 128) * 129 // 128 if case["f8"] else 0) + 4) + 4 * c, "flops": 6 * n * c}
    if op == "norm_grad":
        n, c = case["workers"] * case["rows"], case["cols"]
        return {"bytes": n * (c * SIZE[case["x"]] * (4 if case["residual"] else 3) + 4) + 4 * c
                + case["workers"] * c * SIZE[case["grad"]], "flops": 10 * n * c}
    n = case["workers"] * sum(_counts(case["sizes"]))
    # each gradient is read for the norm and, all of them being known only then, once more
    return {"bytes": 3 * n * SIZE[case["x"]], "flops": 3 * n}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _targets(case, g):
    """Token numbers whose frequency falls as one over their rank, as words' does."""
    workers = case.get("workers", 1)
    u = torch.rand(workers, case["tokens"], generator=g, device=DEV, dtype=torch.float64)
    ids = (float(case["vocab"] + 1) ** u).long().sub(1).clamp(0, case["vocab"] - 1)
    if case["pad"]:  # the tail of each worker's batch
        keep = torch.rand(workers, 1, generator=g, device=DEV) * 0.3 + 0.7
        at = torch.arange(case["tokens"], device=DEV)
        ids = torch.where(at < (keep * case["tokens"]).ceil(), ids, -1)
    return ids.to(TYPES[case["ids"]])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    op, s = case["op"], {"case": case}
    if op in ("loss", "loss_grad"):
        w, t, v, c = case.get("workers", 1), case["tokens"], case["vocab"], case["cols"]
        s["targets"] = _targets(case, g)
        # a final norm's output, and weights whose logits are spread by about 1.5
        s["x"] = normal(w, t, c).to(TYPES[case["x"]])
        s["w"] = (normal(v, c) * (1.5 / math.sqrt(c))).to(TYPES[case["w"]])
        s["loss"], s["lse"] = torch.empty(w, t, device=DEV), torch.empty(w, t, device=DEV)
        if op == "loss_grad":
            # each worker's mean over the tokens that it has
            there = (s["targets"] >= 0).float()
            s["dloss"] = (there / there.sum(-1, keepdim=True)).contiguous()
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty(w, v, c, dtype=TYPES[case["grad"]], device=DEV)
            if case["add"]:  # what the embedding that shares the table has left there
                s["dw"].normal_(std=1e-3, generator=g)
    elif op in ("norm", "norm_grad"):
        n, c, x = case.get("workers", 1) * case["rows"], case["cols"], TYPES[case["x"]]
        s["gamma"] = 1 + 0.1 * normal(c)
        s["eps"] = 1e-5
        # a residual stream, with columns of different sizes
        stream = (normal(n, c) * (1 + normal(c).square())).to(x)
        if op == "norm":
            s["x"] = normal(n, c).to(x) if case["residual"] else stream
            s["residual"] = stream if case["residual"] else None
            s["h"] = torch.empty(n, c, dtype=x, device=DEV) if case["residual"] else None
            s["y"] = torch.empty(n, c, dtype=x, device=DEV) if case["y"] else None
            s["rstd"] = torch.empty(n, device=DEV)
            if case["f8"]:
                s["q"] = torch.empty(n, _up(c, 128), dtype=TYPES[case["f8"]], device=DEV)
                s["q_scale"] = torch.empty(n, _up(_up(c, 128) // 128, 4), dtype=torch.uint8, device=DEV)
        else:
            s["h"] = stream
            s["rstd"] = torch.rsqrt(stream.float().square().mean(-1) + s["eps"])
            s["dy"] = (normal(n, c) * 1e-3).to(x)
            s["dh"] = (normal(n, c) * 1e-3).to(x) if case["residual"] else None
            s["dx"] = torch.empty(n, c, dtype=x, device=DEV)
            s["dgamma"] = torch.empty(case["workers"], c, dtype=TYPES[case["grad"]], device=DEV)
    else:
        # gradients whose sizes differ from worker to worker and from tensor to tensor; what they are
        # clipped into lies side by side in one buffer, as a step's stacks do
        w, x, counts = case["workers"], TYPES[case["x"]], _counts(case["sizes"])
        sizes = torch.exp(normal(len(counts), w, 1)) * 1e-3
        s["grads"] = [normal(w, n).mul_(sizes[i]).to(x) for i, n in enumerate(counts)]
        at = [0]
        for n in counts:
            at.append(at[-1] + _up(w * n, 8))
        s["clipped"] = torch.zeros(at[-1], dtype=x, device=DEV)
        s["outs"] = [s["clipped"][at[i]:at[i] + w * n].view(w, n) for i, n in enumerate(counts)]
        s["norms"] = torch.empty(w, device=DEV)
    return s


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _call(s):
    import sign_muon_step_amd as sm

    case = s["case"]
    op = case["op"]
    if op in ("loss", "loss_grad"):
        if "ws" not in s:
            kinds = (s["x"].dtype, s["w"].dtype)
            s["ws"] = sm.bytes_tensor(sm.signmuon_linear_cross_entropy_workspace_bytes(
                s["targets"].numel(), case["vocab"], case["cols"], *kinds), DEV)
            if op == "loss_grad":
                s["ws_grad"] = sm.bytes_tensor(sm.signmuon_linear_cross_entropy_backward_workspace_bytes(
                    case["workers"], case["tokens"], case["vocab"], case["cols"], *kinds, s["dw"].dtype), DEV)
        sm.signmuon_linear_cross_entropy(s["x"], s["w"], s["targets"], case["scale"], s["loss"], s["lse"], s["ws"])
        if op == "loss":
            return {"loss": s["loss"], "lse": s["lse"]}
        sm.signmuon_linear_cross_entropy_backward(s["x"], s["w"], s["targets"], case["scale"], s["lse"], s["dloss"],
                                                  s["dx"], s["dw"], s["ws_grad"], accumulate=case["add"])
        return {"loss": s["loss"], "lse": s["lse"], "dx": s["dx"], "dw": s["dw"]}
    if op == "norm":
        sm.signmuon_rms_norm(s["x"], s["residual"], s["gamma"], s["eps"], h=s["h"], y=s["y"], q=s.get("q"),
                             q_scale=s.get("q_scale"), rstd=s["rstd"])
        return _normed(s)
    if op == "norm_grad":
        if "ws" not in s:
            s["ws"] = sm.bytes_tensor(sm.signmuon_rms_norm_workspace_bytes(case["workers"], case["rows"], case["cols"]),
                                      DEV)
        sm.signmuon_rms_norm_backward(s["dy"], s["dh"], s["h"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["ws"],
                                      workers=case["workers"])
        return {"dx": s["dx"], "dgamma": s["dgamma"]}
    if "gradients" not in s:
        s["gradients"] = sm.Gradients(s["grads"], s["outs"])
        s["ws"] = sm.bytes_tensor(sm.signmuon_grad_norm_workspace_bytes(s["gradients"]), DEV)
    sm.signmuon_clip_grads(s["gradients"], case["most"], s["norms"], s["ws"])
    return {"norms": s["norms"], "clipped": s["clipped"]}


def _normed(s):
    out = {k: s[k] for k in ("h", "y", "rstd") if s.get(k) is not None}
    if s["case"]["f8"]:  # a scale byte b stands for 2^(b - 127)
        out |= {"q": s["q"], "q_scale": s["q_scale"].view(torch.float8_e8m0fnu)}
    return out


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _quant(x, f8):
    """x [n][k] in blocks of 128 along k: values times 2^-e, rounded to f8, and the bytes e + 127.
    e is the least exponent whose block fits the format (at least -127; 0 for a block of zeros).
    Rows are padded with zeros to a multiple of 128, scales with byte 127 to a multiple of 4."""
    k = x.shape[-1]
    kp, blocks = _up(k, 128), _up(_up(k, 128) // 128, 4)
    x = torch.nn.functional.pad(x, (0, kp - k)).unflatten(-1, (kp // 128, 128))
    top = x.abs().amax(-1)
    m, p = torch.frexp(top)
    e = torch.where(top > 0, (p + (m > 0.875).int() - TOP[f8]).clamp(min=-127), 0)
    q = torch.ldexp(x, -e.unsqueeze(-1)).flatten(-2).to(TYPES[f8])
    return q, torch.nn.functional.pad((e + 127).to(torch.uint8), (0, blocks - kp // 128), value=127)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("loss", "loss_grad"):
        v, c = case["vocab"], case["cols"]
        x, w, ids = s["x"].float().view(-1, c), s["w"].float(), s["targets"].long()
        there, at = (ids >= 0) & (ids < v), ids.clamp(0, v - 1).view(-1, 1)
        logits = torch.matmul(x, w.t()) * case["scale"]
        target = logits.gather(1, at).view_as(ids)
        top = logits.amax(-1, keepdim=True)
        p = logits.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        lse = (top + total.log()).view_as(ids)
        out = {"loss": torch.where(there, lse - target, 0.0), "lse": lse}
        if op == "loss":
            return out
        # dlogits = scale dloss (p - 1 at the target), nothing where there is no target
        d = torch.where(there, s["dloss"] * case["scale"], 0.0).view(-1, 1)
        p.mul_(d / total)
        p.scatter_add_(1, at, -d)
        out["dx"] = torch.matmul(p, w).view_as(s["x"]).to(s["x"].dtype)
        dw = torch.matmul(p.view(case["workers"], -1, v).transpose(1, 2), x.view(case["workers"], -1, c))
        s["dw"].copy_(s["dw"].float() + dw if case["add"] else dw)
        return out | {"dw": s["dw"]}
    if op == "norm":
        # the sum as the residual stream holds it is what is normed
        x = s["x"].float() if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype).float()
        rstd = torch.rsqrt(x.square().mean(-1) + s["eps"])
        y = x * rstd.unsqueeze(-1) * s["gamma"]
        s["rstd"].copy_(rstd)
        if s["h"] is not None:
            s["h"].copy_(x)
        if s["y"] is not None:
            s["y"].copy_(y)
        if case["f8"]:
            s["q"], s["q_scale"] = _quant(y, case["f8"])
        return _normed(s)
    if op == "norm_grad":
        dy, w, c = s["dy"].float(), case["workers"], case["cols"]
        xhat = s["h"].float() * s["rstd"].unsqueeze(-1)
        t = dy * s["gamma"]
        dx = (t - xhat * (t * xhat).mean(-1, keepdim=True)) * s["rstd"].unsqueeze(-1)
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dgamma": (dy * xhat).view(w, -1, c).sum(1).to(s["dgamma"].dtype)}
    squares = torch.stack([x.float().square().sum(-1, dtype=torch.float64) for x in s["grads"]])
    norms = squares.sum(0).sqrt()
    factor = (case["most"] / norms).clamp(max=1.0).float().unsqueeze(-1)
    [out.copy_(x.float() * factor) for x, out in zip(s["grads"], s["outs"])]
    return {"norms": norms.float(), "clipped": s["clipped"]}


def run(state):
    if own:
        return _call(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# In 64 bits
# ---------------------------------------------------------------------------
def _scaled(x, f8):
    """x over its blocks' scales 2^e, and the scales."""
    n, c = x.shape[-1], _up(x.shape[-1], 128)
    out = torch.zeros(x.shape[0], c, dtype=torch.float64, device=x.device)
    out[:, :n] = x
    out = out.unflatten(-1, (-1, 128))
    largest = out.abs().amax(-1, keepdim=True)
    top = 0.875 * 2.0 ** TOP[f8]
    e = torch.ceil(torch.log2(largest / top))
    e = torch.where(largest > torch.exp2(e) * top, e + 1, e)
    e = torch.where(largest <= torch.exp2(e - 1) * top, e - 1, e)
    e = torch.where(largest > 0, e.clamp(min=-127), 0.0)
    scale = torch.exp2(e)
    mantissa, smallest = {"e4m3": (3, -6), "e5m2": (2, -14)}[f8]
    out = (out / scale).flatten(-2)
    step = torch.exp2(torch.floor(torch.log2(out.abs().clamp(min=2.0 ** -40))).clamp(min=smallest) - mantissa)
    return torch.round(out / step) * step, scale.squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op in ("loss", "loss_grad"):
        w, v, c = case.get("workers", 1), case["vocab"], case["cols"]
        loss, lse, dx, dw = [], [], [], []
        table = s["w"].to(f64)
        for i in range(w):  # one worker after the other; a last column takes the padding's targets
            ids = s["targets"][i].long()
            some = (ids >= 0) & (ids < v)
            x = s["x"][i].to(f64)
            logits = case["scale"] * (x @ table.T.contiguous())
            lse.append(torch.logsumexp(logits, dim=1))
            rows = torch.arange(ids.numel(), device=DEV)
            at = torch.where(some, ids, 0)
            loss.append((lse[-1] - logits[rows, at]) * some)
            if op == "loss_grad":
                g = torch.softmax(logits, dim=1)
                g[rows[some], ids[some]] -= 1
                g *= (case["scale"] * s["dloss"][i].to(f64) * some)[:, None]
                dx.append(g @ table)
                dw.append(g.T.contiguous() @ x)
        out = {"loss": torch.stack(loss), "lse": torch.stack(lse)}
        if op == "loss":
            return out
        dw = torch.stack(dw)
        return out | {"dx": torch.stack(dx), "dw": dw + s["dw"].to(f64) if case["add"] else dw}
    if op == "norm":
        total = s["x"].to(f64) if s["residual"] is None else s["x"].to(f64) + s["residual"].to(f64)
        x = total.to(torch.float32).to(s["x"].dtype).to(f64)
        rstd = 1 / torch.sqrt((x * x).mean(-1) + s["eps"])
        y = x * rstd[:, None] * s["gamma"].to(f64)
        out = {"rstd": rstd}
        if s["h"] is not None:
            out["h"] = total
        if case["y"]:
            out["y"] = y
        if case["f8"]:
            out["q"], scale = _scaled(y, case["f8"])
            out["q_scale"] = torch.ones(s["q_scale"].shape, dtype=f64, device=DEV)
            out["q_scale"][:, : scale.shape[1]] = scale
        return out
    if op == "norm_grad":
        w, c = case["workers"], case["cols"]
        dy, gamma, rstd = s["dy"].to(f64), s["gamma"].to(f64), s["rstd"].to(f64)[:, None]
        xhat = s["h"].to(f64) * rstd
        t = dy * gamma
        # the share of t along xhat, of squared length c, falls out of the gradient
        dx = rstd * (t - xhat * ((t * xhat).sum(-1, keepdim=True) / c))
        return {"dx": dx if s["dh"] is None else dx + s["dh"].to(f64), "dgamma": (dy * xhat).view(w, -1, c).sum(1)}
    norms = torch.stack([torch.stack([torch.linalg.vector_norm(x[m], dtype=f64) for x in s["grads"]]).norm()
                         for m in range(case["workers"])])
    factor = torch.where(norms > case["most"], case["most"] / norms, 1.0)
    clipped = torch.zeros(s["clipped"].shape, dtype=f64, device=DEV)
    at = 0
    for x in s["grads"]:
        clipped[at:at + x.numel()] = (x.to(f64) * factor[:, None]).flatten()
        at += _up(x.numel(), 8)
    return {"norms": norms, "clipped": clipped}
