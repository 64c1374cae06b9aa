"""Root-mean-square norm with the residual's addition, its 8-bit output and its
gradients against a plain implementation in 64 bits.

Tolerances count roundings, with u = 2^-24. A sum of n terms added in a tree of
depth d and chains of length l is off by at most (d + l) u times the sum of the
terms' sizes."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, TINY, Guarded, replays_like_eager, same_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 3, -6), "e5m2": (torch.float8_e5m2, 57344.0, 2, -14)}


@pytest.fixture(autouse=True)
def _name_the_case(request):
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()


def depth(cols):
    """Additions that one value of a row's sum goes through, at most: a lane's
    own chain, a wave's tree, the waves' chain."""
    lane = 32 if cols <= 16384 else 8 * ((cols + 8191) // 8192)
    return lane + 6 + 16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inputs(rows, cols, dtype, seed):
    x = torch.randn(rows, cols, generator=gen(seed)).to(dtype)
    # rows of very different sizes, as a residual stream's are
    r = (torch.randn(rows, cols, generator=gen(seed + 1)) * torch.exp(torch.randn(rows, 1, generator=gen(seed + 2)))).to(dtype)
    gamma = 1 + 0.3 * torch.randn(cols, generator=gen(seed + 3))
    return x, r, gamma


def stored_sum(x, r):
    """x + r in fp32, rounded to the type: what h holds, bit for bit."""
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def normed(h, gamma, eps):
    """In 64 bits: rstd and y, and how far fp32 may be off in each."""
    h, cols = h.double(), h.shape[-1]
    eps = float(torch.tensor(eps, dtype=torch.float32))
    square = h.square().mean(-1)
    rstd = 1 / torch.sqrt(square + eps)
    # the squares and their sum (d + 1), 1 / cols and the product (2), eps (1): halved by the root;
    # root and quotient
    rel = 0.5 * (depth(cols) + 4) * U + 4 * U
    y = h * rstd[:, None] * gamma.double()
    return rstd, rel * rstd, y, (rel + 3 * U) * y.abs()


SIZES = [(1, 1), (3, 2), (5, 7), (9, 63), (8, 64), (7, 65), (13, 128), (4, 129), (100, 255), (6, 257), (17, 512),
         (5, 513), (100, 769), (33, 1023), (3, 1025), (5, 1536), (2, 2047), (6, 2049), (1, 4096), (5, 4100),
         (2, 8191), (3, 9000), (2, 16384), (3, 16385), (2, 40001)]


def run_forward(x, r, gamma, eps, f8=None, y=True, keep=True):
    rows, cols = x.shape
    out = {"rstd": Guarded((rows,), torch.float32)}
    if r is not None and keep:
        out["h"] = Guarded((rows, cols), x.dtype)
    if y:
        out["y"] = Guarded((rows, cols), x.dtype)
    if f8:
        out["q"] = Guarded((rows, sm.signmuon_f8_pitch(cols)), F8[f8][0])
        out["q_scale"] = Guarded((rows, sm.signmuon_f8_scale_pitch(cols)), torch.uint8)
    sm.signmuon_rms_norm(x.to(DEV), None if r is None else r.to(DEV), gamma.to(DEV), eps,
                         **{k: o.t for k, o in out.items()})
    torch.cuda.synchronize()
    for k, o in out.items():
        o.check(k)
    return {k: o.t for k, o in out.items()}


def check_f8(q, scale, y, y_tol, f8):
    """q and its scales stand for y, off by y_tol, rounded to the format."""
    dtype, top, mantissa, smallest = F8[f8]
    rows, cols = y.shape
    blocks = (cols + 127) // 128
    assert bool((q.view(torch.uint8)[:, cols:] == 0).all()) and bool((scale[:, blocks:] == 127).all())
    pad = torch.nn.functional.pad
    by = lambda v: pad(v, (0, blocks * 128 - cols)).unflatten(-1, (blocks, 128))  # noqa: E731
    y, y_tol = by(y), by(y_tol)
    s = torch.exp2(scale.cpu()[:, :blocks].double() - 127)[:, :, None]
    size, off = y.abs().amax(-1, keepdim=True), y_tol.amax(-1, keepdim=True)
    assert bool((size <= s * top * 1.0000001 + off).all()), "a scale too small"
    assert bool(((size > s / 2 * top - off) | (size == 0)).all()), "a scale too large"
    got = q.cpu().float().double().unflatten(-1, (blocks, 128)) * s
    step = torch.exp2(torch.floor(torch.log2((y.abs() + y_tol) / s).clamp(min=smallest)) - mantissa) * s
    assert bool(((got - y).abs() <= step / 2 + y_tol + TINY).all())


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("f8", [None, "e4m3", "e5m2"])
def test_forward(rows, cols, dtype, residual, f8):
    eps = 1e-5
    x, r, gamma = inputs(rows, cols, dtype, rows + cols)
    r = r if residual else None
    h = stored_sum(x, r)
    got = run_forward(x, r, gamma, eps, f8)
    if residual:
        assert same_bits(got["h"].cpu(), h)
    rstd, rstd_tol, y, y_tol = normed(h, gamma, eps)
    assert bool(((got["rstd"].cpu().double() - rstd).abs() <= 1.01 * rstd_tol).all())
    tol = 1.01 * y_tol + HALF_STEP[dtype] * (y.abs() + 1.01 * y_tol) + TINY
    assert bool(((got["y"].cpu().double() - y).abs() <= tol).all())
    if f8:
        check_f8(got["q"], got["q_scale"], y, 1.01 * y_tol, f8)


@pytest.mark.parametrize("cols", [40, 515, 4096, 12000, 20000])
@pytest.mark.parametrize("f8", ["e4m3", "e5m2"])
def test_the_8_bit_output_is_that_of_the_quantisation(cols, f8):
    """In fp32 the output y is what is quantised: the same bytes as quantising y."""
    x, r, gamma = inputs(21, cols, torch.float32, cols)
    got = run_forward(x, r, gamma, 1e-6, f8)
    q, scale = sm.f8_empty((21, cols), F8[f8][0], DEV)
    sm.signmuon_f8_quant(got["y"], q, scale)
    assert same_bits(q, got["q"]) and same_bits(scale, got["q_scale"])
    alone = run_forward(x, r, gamma, 1e-6, f8, y=False, keep=False)
    assert same_bits(q, alone["q"]) and same_bits(scale, alone["q_scale"]) and same_bits(alone["rstd"], got["rstd"])


@pytest.mark.parametrize("cols", [1, 100, 768, 1111, 5000, 9001, 17000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_sum_in_place_of_either_addend(cols, dtype):
    x, r, gamma = (t.to(DEV) for t in inputs(37, cols, dtype, 3 * cols))
    want = {k: torch.empty_like(x) for k in "hy"}
    sm.signmuon_rms_norm(x, r, gamma, 1e-5, **want)
    for at in (0, 1):
        a, y = [x.clone(), r.clone()], torch.empty_like(x)
        sm.signmuon_rms_norm(*a, gamma, 1e-5, h=a[at], y=y)
        assert same_bits(a[at], want["h"]) and same_bits(y, want["y"]) and same_bits(a[1 - at], (r, x)[at])


def test_extreme_rows_stay_their_own():
    rows, cols = 9, 300
    x = torch.randn(rows, cols, generator=gen(1))
    x[1, 7], x[3, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    x[5], x[6], x[7] = 0.0, 1e-30, 3e38
    x = x.to(DEV)
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    q, scale = sm.f8_empty((rows, cols), torch.float8_e4m3fn, DEV)
    q.view(torch.uint8).fill_(0x55)
    sm.signmuon_rms_norm(x, None, torch.ones(cols, device=DEV), 1e-5, y=y, q=q, q_scale=scale, rstd=rstd)
    torch.cuda.synchronize()
    assert y[[0, 2, 5, 6, 7, 8]].isfinite().all() and y[[1, 3, 4]].isnan().any(-1).all()
    assert bool((y[5] == 0).all()) and bool((scale[5] == 127).all())
    # squares past fp32: the output is 0, as the header says
    assert bool((y[7] == 0).all()) and float(rstd[7]) == 0
    assert bool((q.view(torch.uint8)[:, cols:] == 0).all())
    assert q.float()[[0, 2, 5, 6, 7, 8]].isfinite().all()


# ---------------------------------------------------------------------------
# Backward
# ---------------------------------------------------------------------------
def backward_in_64(dy, dh, h, gamma, rstd, workers):
    """The gradients from the given statistics, and their tolerances."""
    cols = h.shape[-1]
    dy, h, g, r = dy.double(), h.double(), gamma.double(), rstd.double()[:, None]
    xh, t = h * r, dy * g
    along = (t * xh).mean(-1, keepdim=True)
    own = r * (t - xh * along)
    dx = own if dh is None else own + dh.double()
    # products of t (u) and xh (u), their sum (d + 1) and the mean (2)
    along_tol = (depth(cols) + 5) * U * (t * xh).abs().mean(-1, keepdim=True)
    # t: u, xh along: 2 u, difference and the product with rstd: 2 u of the two parts; dh's addition
    dx_tol = r * (xh.abs() * along_tol + U * (3 * t.abs() + 5 * (xh * along).abs())) + U * dx.abs()
    rows = h.shape[0] // workers
    by = lambda v: v.view(workers, rows, cols).sum(1)  # noqa: E731
    # a column's chain: at most every row of the worker, then trees
    return dx, dx_tol, by(dy * xh), (rows + 24 + 2) * U * by((dy * xh).abs())


BACKWARD = [(1, 1, 1), (1, 5, 2), (2, 3, 9), (3, 40, 63), (1, 65, 64), (2, 33, 100), (5, 70, 129), (1, 100, 256),
            (2, 37, 500), (3, 111, 515), (8, 40, 768), (1, 9, 1024), (2, 50, 1111), (1, 70, 2048), (2, 9, 2049),
            (1, 5, 4095), (2, 3, 5000), (1, 6, 8192), (1, 7, 16383), (2, 19, 16390), (1, 40, 30001)]


def run_backward(dy, dh, h, gamma, rstd, workers, grad_dtype, want=(True, True)):
    rows, cols = h.shape
    dx, dg = Guarded((rows, cols), h.dtype), Guarded((workers, cols), grad_dtype)
    ws = Guarded((sm.signmuon_rms_norm_workspace_bytes(workers, rows // workers, cols),), torch.uint8)
    outs = [o.t if w else None for o, w in zip((dx, dg), want)]
    sm.signmuon_rms_norm_backward(dy.to(DEV), None if dh is None else dh.to(DEV), h.to(DEV), gamma.to(DEV),
                                  rstd.to(DEV), *outs, ws.t if ws.nbytes else None, workers=workers)
    torch.cuda.synchronize()
    for o, name in ((dx, "dx"), (dg, "dgamma"), (ws, "workspace")):
        o.check(name)
    return outs


def backward_inputs(workers, rows, cols, dtype, seed):
    n = workers * rows
    _, h, gamma = inputs(n, cols, dtype, seed)
    dy = torch.randn(n, cols, generator=gen(seed + 5)).to(dtype)
    dh = torch.randn(n, cols, generator=gen(seed + 6)).to(dtype)
    return dy, dh, h, gamma, normed(h, gamma, 1e-5)[0].float()


@pytest.mark.parametrize("workers,rows,cols", BACKWARD)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("stream", [False, True])
def test_backward(workers, rows, cols, dtype, grad_dtype, stream):
    dy, dh, h, gamma, rstd = backward_inputs(workers, rows, cols, dtype, rows * cols + workers)
    dh = dh if stream else None
    got = run_backward(dy, dh, h, gamma, rstd, workers, grad_dtype)
    want = backward_in_64(dy, dh, h, gamma, rstd, workers)
    for g, w, tol, name in zip(got, want[::2], want[1::2], ("dx", "dgamma")):
        tol = 1.01 * tol + HALF_STEP[g.dtype] * (w.abs() + tol) + TINY
        assert bool(((g.cpu().double() - w).abs() <= tol).all()), name


@pytest.mark.parametrize("cols", [60, 768, 3000, 17000])
def test_backward_of_some_outputs_only_and_in_place(cols):
    workers, rows = 2, 50
    dy, dh, h, gamma, rstd = backward_inputs(workers, rows, cols, torch.bfloat16, 3)
    args = (dy, dh, h, gamma, rstd, workers, torch.float32)
    whole = run_backward(*args)
    for want in [(True, False), (False, True)]:
        for g, w in zip(run_backward(*args, want=want), whole):
            assert g is None or same_bits(g, w)
    ws = sm.bytes_tensor(sm.signmuon_rms_norm_workspace_bytes(workers, rows, cols), DEV)
    for at in (0, 1):
        d = [dy.to(DEV), dh.to(DEV)]
        dgamma = torch.empty(workers, 1, cols, device=DEV)
        sm.signmuon_rms_norm_backward(*d, h.to(DEV), gamma.to(DEV), rstd.to(DEV), d[at], dgamma, ws, workers=workers)
        assert same_bits(d[at], whole[0]) and same_bits(dgamma.view(workers, cols), whole[1])
        assert same_bits(d[1 - at].cpu(), (dh, dy)[at])


def test_backward_is_the_forwards_by_differences():
    """Central differences of a weighted sum of both outputs (h and y), along one
    direction of x and gamma, in 64 bits, against the kernel's gradients."""
    rows, cols, eps, step = 12, 200, 1e-5, 1e-4
    x, r, gamma = inputs(rows, cols, torch.float32, 77)
    dy, dh = (torch.randn(rows, cols, generator=gen(78 + i)) for i in (0, 1))
    dirs = [torch.randn(s, generator=gen(80 + i), dtype=torch.float64) for i, s in enumerate(((rows, cols), (cols,)))]
    got = run_forward(x, r, gamma, eps)
    grads = run_backward(dy, dh, got["h"], gamma, got["rstd"], 1, torch.float32)

    def loss(t):
        h, g = x.double() + r.double() + t * dirs[0], gamma.double() + t * dirs[1]
        y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * g
        return float((y * dy.double()).sum() + (h * dh.double()).sum())

    by_difference = (loss(step) - loss(-step)) / (2 * step)
    by_gradient = sum(float((g.cpu().double().view(-1) * d.view(-1)).sum()) for g, d in zip(grads, dirs))
    # step^2 of the third derivative, and 2400 products off by a few u each
    assert abs(by_difference - by_gradient) < 1e-4 * rows * cols * step + 1e-3


def test_replays_and_streams_give_the_same_bits():
    workers, rows, cols = 3, 200, 515
    x, r, gamma = (t.to(DEV) for t in inputs(workers * rows, cols, torch.bfloat16, 4))
    dy, dh, h, y, dx = (torch.empty_like(x) for _ in range(5))
    rstd, dg = torch.empty(workers * rows, device=DEV), torch.empty(workers, 1, cols, device=DEV)
    q, scale = sm.f8_empty(x.shape, torch.float8_e4m3fn, DEV)
    ws = sm.bytes_tensor(sm.signmuon_rms_norm_workspace_bytes(workers, rows, cols), DEV)

    def refresh(i):
        a, b, _ = inputs(workers * rows, cols, torch.bfloat16, 40 + 7 * i)
        x.copy_(a), r.copy_(b)
        dy.copy_(torch.randn(workers * rows, cols, generator=gen(50 + i)))
        dh.copy_(torch.randn(workers * rows, cols, generator=gen(60 + i)))

    def call(stream=None):
        sm.signmuon_rms_norm(x, r, gamma, 1e-5, h=h, y=y, q=q, q_scale=scale, rstd=rstd, stream=stream)
        sm.signmuon_rms_norm_backward(dy, dh, h, gamma, rstd, dx, dg, ws, workers=workers, stream=stream)

    outs = [h, y, q, scale, rstd, dx, dg]
    replays_like_eager(call, outs, refresh)
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    call(torch.cuda.Stream())
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert same_bits(a, b)
