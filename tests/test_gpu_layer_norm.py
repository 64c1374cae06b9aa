"""Layer norm and its gradients against a plain implementation in 64 bits.

Tolerances count roundings, with u = 2^-24. A sum of n terms added in a tree of
depth d and chains of length l is off by at most (d + l) u times the sum of the
terms' sizes; the longest chain here is DEPTH. The statistics' errors then
follow from their formulas (written beside each)."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, TINY, Guarded, replays_like_eager, same_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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


def inputs(rows, cols, dtype, seed, offset=0.5):
    x = torch.randn(rows, cols, generator=gen(seed)) * 2 + offset
    gamma = 1 + 0.3 * torch.randn(cols, generator=gen(seed + 1))
    beta = 0.2 * torch.randn(cols, generator=gen(seed + 2))
    return x.to(dtype), gamma, beta


def statistics(x, eps):
    """In 64 bits: mean, rstd, and how far fp32 sums may be off in each."""
    x, n, d = x.double(), x.shape[-1], depth(x.shape[-1])
    mean = x.mean(-1)
    mean_tol = (d + 3) * U * x.abs().mean(-1)  # the sum, 1 / cols and the product
    var = x.var(-1, unbiased=False)
    # differences to a mean that is off by m: their squares' mean grows by m^2; each difference is
    # rounded (u |x - mean|), squared and added (2 u + d u of the square)
    var_tol = mean_tol ** 2 + 2 * U * (x - mean[:, None]).abs().pow(2).mean(-1) * (d + 6)
    rstd = 1 / torch.sqrt(var + eps)
    # d rstd = -rstd / 2 * d var / (var + eps), and sqrt, division and the sum of eps
    rstd_tol = rstd * (0.5 * var_tol / (var + eps) + 4 * U)
    return mean, mean_tol, rstd, rstd_tol


SIZES = [(1, 1), (3, 2), (5, 7), (9, 63), (8, 64), (7, 65), (13, 128), (4, 129), (100, 255), (6, 257), (17, 512),
         (5, 513), (100, 769), (33, 1023), (3, 1025), (5, 1536), (2, 2047), (6, 2049), (3, 4096), (5, 4100),
         (2, 8191), (3, 9000), (2, 16384), (3, 16385), (2, 40001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bias", [False, True])
def test_forward(rows, cols, dtype, bias):
    eps = 1e-5
    x, gamma, beta = inputs(rows, cols, dtype, rows + cols)
    y, mean, rstd = Guarded((rows, cols), dtype), Guarded((rows,), torch.float32), Guarded((rows,), torch.float32)
    sm.signmuon_layer_norm(x.to(DEV), gamma.to(DEV), beta.to(DEV) if bias else None, eps, y.t, mean.t, rstd.t)
    torch.cuda.synchronize()
    for o, name in ((y, "y"), (mean, "mean"), (rstd, "rstd")):
        o.check(name)
    eps32 = float(torch.tensor(eps, dtype=torch.float32))
    m, m_tol, r, r_tol = statistics(x, eps32)
    assert bool(((mean.t.cpu().double() - m).abs() <= m_tol + TINY).all())
    assert bool(((rstd.t.cpu().double() - r).abs() <= r_tol).all())
    g = gamma.double()
    scaled = (x.double() - m[:, None]) * r[:, None] * g
    want = scaled + (beta.double() if bias else 0.0)
    # the difference (m_tol, u), times rstd (r_tol, u), times gamma plus beta (u)
    tol = m_tol[:, None] * (r[:, None] * g).abs() + scaled.abs() * ((r_tol / r)[:, None] + 3 * U) + U * want.abs()
    tol = 1.01 * tol + HALF_STEP[dtype] * (want.abs() + tol) + TINY
    assert bool(((y.t.cpu().double() - want).abs() <= tol).all())


def test_forward_without_statistics_and_with_far_means():
    for cols in (48, 700, 3000, 20000):
        x, gamma, beta = inputs(20, cols, torch.float32, cols, offset=1000.0)
        y, z = torch.empty(20, cols, device=DEV), torch.empty(20, cols, device=DEV)
        mean, rstd = torch.empty(20, device=DEV), torch.empty(20, device=DEV)
        sm.signmuon_layer_norm(x.to(DEV), gamma.to(DEV), beta.to(DEV), 1e-5, y)
        sm.signmuon_layer_norm(x.to(DEV), gamma.to(DEV), beta.to(DEV), 1e-5, z, mean, rstd)
        assert same_bits(y, z)
        _, _, r, r_tol = statistics(x, 1e-5)
        # a variance from squares would have lost 1000^2 / 4 * u of itself here
        assert bool(((rstd.cpu().double() - r).abs() <= r_tol + 1e-12).all())


def test_forward_of_a_row_of_equal_values():
    x = torch.full((3, 700), 4.0, device=DEV)  # sums of 4 are exact
    gamma, beta = torch.randn(700, device=DEV), torch.randn(700, device=DEV)
    y, rstd = torch.empty_like(x), torch.empty(3, device=DEV)
    sm.signmuon_layer_norm(x, gamma, beta, 1e-2, y, None, rstd)
    # the mean is off by u of 4 at most, times rstd = 10
    assert bool(((y - beta).abs() <= 4 * 12 * U * 10 * gamma.abs() + U).all())
    assert bool(((rstd - 10).abs() < 1e-5).all())


def test_nan_and_infinity_stay_in_their_row():
    x = torch.randn(6, 300, device=DEV)
    x[1, 7], x[3, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    gamma = torch.ones(300, device=DEV)
    y = torch.empty_like(x)
    sm.signmuon_layer_norm(x, gamma, None, 1e-5, y)
    assert y[[0, 2, 5]].isfinite().all() and y[[1, 3, 4]].isnan().any(-1).all()


def backward_in_64(dy, x, gamma, mean, rstd, workers):
    """The three gradients from the given statistics, and their tolerances."""
    cols = x.shape[-1]
    dy, x, g, r = dy.double(), x.double(), gamma.double(), rstd.double()[:, None]
    d = depth(cols)
    xh = (x - mean.double()[:, None]) * r
    t = dy * g
    s1, s2 = t.mean(-1, keepdim=True), (t * xh).mean(-1, keepdim=True)
    dx = r * (t - s1 - xh * s2)
    # t: u; xh: 2 u; each sum: d u and 2 u for the mean, of its sizes
    s1_tol = (d + 4) * U * t.abs().mean(-1, keepdim=True)
    s2_tol = (d + 6) * U * (t * xh).abs().mean(-1, keepdim=True)
    dx_tol = r * (s1_tol + xh.abs() * s2_tol + U * (4 * t.abs() + 3 * s1.abs() + 7 * (xh * s2).abs()))
    rows = x.shape[0] // workers
    by = lambda v: v.view(workers, rows, cols).sum(1)  # noqa: E731
    # a column's chain: at most every row of the worker, then trees
    chain = rows + 24
    return (dx, dx_tol, by(dy * xh), (chain + 3) * U * by((dy * xh).abs()), by(dy), chain * U * by(dy.abs()))


BACKWARD = [(1, 1, 1), (1, 5, 2), (2, 3, 9), (3, 40, 63), (1, 65, 64), (2, 33, 100), (5, 70, 129), (1, 100, 256),
            (2, 37, 500), (3, 111, 515), (8, 40, 768), (1, 9, 1024), (2, 50, 1111), (1, 70, 2048), (2, 9, 2049),
            (1, 5, 4095), (2, 3, 5000), (1, 6, 8192), (1, 7, 16383), (2, 19, 16390), (1, 40, 30001)]


def run_backward(dy, x, gamma, mean, rstd, workers, grad_dtype, want=(True, True, True)):
    rows, cols = x.shape
    dx = Guarded((rows, cols), x.dtype)
    dg, db = Guarded((workers, cols), grad_dtype), Guarded((workers, cols), grad_dtype)
    ws = Guarded((sm.signmuon_layer_norm_workspace_bytes(workers, rows // workers, cols),), torch.uint8)
    outs = [o.t if w else None for o, w in zip((dx, dg, db), want)]
    sm.signmuon_layer_norm_backward(dy.to(DEV), x.to(DEV), gamma.to(DEV), mean.to(DEV), rstd.to(DEV), *outs,
                                    ws.t if ws.nbytes else None, workers=workers)
    torch.cuda.synchronize()
    for o, name in ((dx, "dx"), (dg, "dgamma"), (db, "dbeta"), (ws, "workspace")):
        o.check(name)
    return outs


@pytest.mark.parametrize("workers,rows,cols", BACKWARD)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
def test_backward(workers, rows, cols, dtype, grad_dtype):
    x, gamma, _ = inputs(workers * rows, cols, dtype, rows * cols + workers)
    dy = torch.randn(workers * rows, cols, generator=gen(5)).to(dtype)
    mean, _, rstd, _ = statistics(x, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    got = run_backward(dy, x, gamma, mean, rstd, workers, grad_dtype)
    want = backward_in_64(dy, x, gamma, mean, rstd, workers)
    for g, w, tol, name in zip(got, want[::2], want[1::2], ("dx", "dgamma", "dbeta")):
        tol = 1.01 * tol + HALF_STEP[g.dtype] * (w.abs() + tol) + TINY
        assert bool(((g.cpu().double() - w).abs() <= tol).all()), name


@pytest.mark.parametrize("cols", [60, 768, 3000, 17000])
def test_backward_of_some_outputs_only(cols):
    workers, rows = 2, 50
    x, gamma, _ = inputs(workers * rows, cols, torch.float32, 3)
    dy = torch.randn(workers * rows, cols, generator=gen(6))
    mean, _, rstd, _ = statistics(x, 1e-5)
    args = (dy, x, gamma, mean.float(), rstd.float(), workers, torch.float32)
    whole = run_backward(*args)
    for want in [(True, False, False), (False, True, False), (False, False, True), (False, True, True),
                 (True, False, True)]:
        for g, w in zip(run_backward(*args, want=want), whole):
            assert g is None or same_bits(g, w)


def test_backward_is_the_forwards_by_differences():
    """Central differences of a weighted sum of the outputs, along one direction
    of x, gamma and beta, computed in 64 bits, against the kernel's gradients."""
    rows, cols, eps, step = 12, 200, 1e-5, 1e-4
    x, gamma, beta = inputs(rows, cols, torch.float32, 77)
    dy = torch.randn(rows, cols, generator=gen(78))
    dirs = [torch.randn(s, generator=gen(79 + i), dtype=torch.float64) for i, s in
            enumerate(((rows, cols), (cols,), (cols,)))]
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    sm.signmuon_layer_norm(x.to(DEV), gamma.to(DEV), beta.to(DEV), eps, torch.empty(rows, cols, device=DEV), mean, rstd)
    grads = run_backward(dy, x, gamma, mean, rstd, 1, torch.float32)

    def loss(h):
        xx, g, b = (v.double() + h * d for v, d in zip((x, gamma, beta), dirs))
        z = (xx - xx.mean(-1, keepdim=True)) / torch.sqrt(xx.var(-1, unbiased=False, keepdim=True) + eps) * g + b
        return float((z * dy.double()).sum())

    by_difference = (loss(step) - loss(-step)) / (2 * step)
    by_gradient = sum(float((g.cpu().double().view(-1) * d.view(-1)).sum()) for g, d in zip(grads, dirs))
    # step^2 of the third derivative, and 2400 products off by a few u each
    assert abs(by_difference - by_gradient) < 1e-4 * rows * cols * step + 1e-3


def test_replays_and_streams_give_the_same_bits():
    workers, rows, cols = 3, 200, 515
    x, gamma, beta = (t.to(DEV) for t in inputs(workers * rows, cols, torch.bfloat16, 4))
    dy = torch.empty_like(x)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(workers * rows, device=DEV), torch.empty(workers * rows, device=DEV)
    dg, db = torch.empty(workers, 1, cols, device=DEV), torch.empty(workers, 1, cols, device=DEV)
    ws = sm.bytes_tensor(sm.signmuon_layer_norm_workspace_bytes(workers, rows, cols), DEV)

    def refresh(i):
        x.copy_(inputs(workers * rows, cols, torch.bfloat16, 40 + i)[0])
        dy.copy_(torch.randn(workers * rows, cols, generator=gen(50 + i)))

    def call(stream=None):
        sm.signmuon_layer_norm(x, gamma, beta, 1e-5, y, mean, rstd, stream=stream)
        sm.signmuon_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dg, db, ws, workers=workers, stream=stream)

    replays_like_eager(call, [y, mean, rstd, dx, dg, db], refresh)
    want = [t.clone() for t in (y, dx, dg, db)]
    torch.cuda.synchronize()
    call(torch.cuda.Stream())
    torch.cuda.synchronize()
    for a, b in zip((y, dx, dg, db), want):
        assert same_bits(a, b)
