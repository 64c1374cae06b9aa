"""Softmax cross entropy of an output layer and its gradients against a plain
implementation in 64 bits.

Tolerances count roundings, with u = 2^-24. Sums on the matrix cores follow the
probabilistic bound for a chain of n roundings (Higham and Mary, SIAM J. Sci.
Comput. 2019): 4 sqrt(n) u times the sum of the terms' sizes. What is held in one
BF16 plane is off by 2^-8 of itself, in two by 2^-16, in three by 2^-24; of a
product of two operands in three planes, pairs of 2^-8 by 2^-16 are left out."""
import math

import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, TINY, Guarded, replays_like_eager, same_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _name_the_case(request):
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, seed, pad=True, ids=torch.int64, spread=2.0):
    x = torch.randn(workers, tokens, cols, generator=gen(seed)).to(x_dtype)
    w = (torch.randn(vocab, cols, generator=gen(seed + 1)) * (spread / math.sqrt(cols))).to(w_dtype)
    targets = torch.randint(0, vocab, (workers, tokens), generator=gen(seed + 2))
    if pad:  # about an eighth, by several kinds of number outside the vocabulary
        outside = torch.tensor([-1, -100, vocab, vocab + 1000, 2 ** 31 - 1, -2 ** 31 if ids == torch.int32 else 2 ** 32 + 3])
        which = torch.randint(0, 48, (workers, tokens), generator=gen(seed + 3))
        targets = torch.where(which < 6, outside[which.clamp(max=5)], targets)
    dloss = torch.randn(workers, tokens, generator=gen(seed + 4))
    return x.to(DEV), w.to(DEV), targets.to(ids).to(DEV), dloss.to(DEV)


def logits_in_64(x, w, scale):
    """Logits, and how far fp32 may be off in each."""
    x, w = x.double().flatten(0, -2), w.double()
    both = x.dtype, w.dtype
    assert both == (torch.float64, torch.float64)
    l, size = scale * (x @ w.t().contiguous()), abs(scale) * (x.abs() @ w.abs().t().contiguous())
    # up to six pairs of planes; what they leave out; factor and product
    return l, (4 * math.sqrt(6 * x.shape[1] + 4) + 4) * U * size + 3 * U * l.abs()


def losses_in_64(l, l_tol, targets, vocab):
    targets = targets.long().flatten()
    there = (targets >= 0) & (targets < vocab)
    lse = torch.logsumexp(l, 1)
    at = torch.where(there, targets, 0)[:, None]
    p = torch.exp(l - lse[:, None])
    # exponents are differences of logits in units of log 2 (2 u of their size), each exponential is off
    # by 2 u, and sums go through a lane's 64, 2 lanes, a wave's share of the blocks and 16 waves
    d = 64 + 2 + vocab / 2048 + 18
    size = l.abs().amax(1)
    lse_tol = (p * l_tol).sum(1) + (d + 4) * U + 4 * U * size + 4 * U * lse.abs()
    loss = torch.where(there, lse - l.gather(1, at)[:, 0], 0.0)
    loss_tol = torch.where(there, lse_tol + l_tol.gather(1, at)[:, 0] + 6 * U * size, 0.0)
    return lse, lse_tol, loss, loss_tol, there


def run_forward(x, w, targets, scale):
    loss, lse = Guarded(tuple(targets.shape), F32), Guarded(tuple(targets.shape), F32)
    ws = Guarded((sm.signmuon_linear_cross_entropy_workspace_bytes(targets.numel(), *w.shape, x.dtype, w.dtype),),
                 torch.uint8)
    sm.signmuon_linear_cross_entropy(x, w, targets, scale, loss.t, lse.t, ws.t)
    torch.cuda.synchronize()
    for o, name in ((loss, "loss"), (lse, "lse"), (ws, "workspace")):
        o.check(name)
    return loss.t, lse.t


def run_backward(x, w, targets, scale, lse, dloss, grad_dtype, start=None, want=(True, True)):
    workers, tokens, cols = x.shape
    vocab = w.shape[0]
    dx, dw = Guarded(tuple(x.shape), x.dtype), Guarded((workers, vocab, cols), grad_dtype)
    if start is not None:
        dw.t.copy_(start)
    ws = Guarded((sm.signmuon_linear_cross_entropy_backward_workspace_bytes(workers, tokens, vocab, cols, x.dtype,
                                                                           w.dtype, grad_dtype),), torch.uint8)
    outs = [o.t if k else None for o, k in zip((dx, dw), want)]
    sm.signmuon_linear_cross_entropy_backward(x, w, targets, scale, lse, dloss, *outs, ws.t,
                                              accumulate=start is not None)
    torch.cuda.synchronize()
    for o, name in ((dx, "dx"), (dw, "dw"), (ws, "workspace")):
        o.check(name)
    return outs


def gradients_in_64(x, w, targets, scale, lse, dloss, grad_dtype, whole_g=False):
    """dx and dw from the given lse, and their tolerances. whole_g: BF16 results of g in three planes."""
    workers, tokens, cols = x.shape
    vocab = w.shape[0]
    l, l_tol = logits_in_64(x, w, scale)
    targets, lse, d = targets.long().flatten(), lse.double().flatten(), dloss.double().flatten()
    there = ((targets >= 0) & (targets < vocab))[:, None]
    p = torch.exp(l - lse[:, None])
    one = torch.zeros_like(p).scatter_(1, targets.clamp(0, vocab - 1)[:, None], 1.0)
    d = (scale * d)[:, None]
    g = torch.where(there, d * (p - one), 0.0)
    # the exponent: the logit, lse in units of log 2 (2 u), the difference (u of both); the exponential 2 u
    p_tol = p * (l_tol + 3 * U * lse.abs()[:, None] + 2 * U * l.abs() + 3 * U)
    g_tol = torch.where(there, d.abs() * p_tol + 3 * U * g.abs(), 0.0)
    x64, w64 = x.double().flatten(0, 1), w.double()

    def product(rows, a, a_tol, b, b_dtype, fp32):
        n = 3 if fp32 or whole_g else 1
        # g; an fp32 operand that meets it (in three planes, or two); two pairs that are left out of three each
        part = 2.0 ** (-8 * n) + (0.0 if b_dtype == BF16 else 3 * 2.0 ** -24 if fp32 else 2.0 ** -16)
        size = a.abs() @ b.abs()
        # a plane's value below 2^-126, BF16's smallest normal one, counts as 0: a factor in n planes is off
        # by 2^-126 for each (an exponential of -88 times a token of 512 is 2^-118, and passes TINY)
        lost = n * 2.0 ** -126 * (b.abs().sum(0) + a.abs().sum(1, keepdim=True))
        return a @ b, 1.01 * (a_tol @ b.abs()) + (1.01 * part + 4 * math.sqrt(6 * rows + 4) * U) * size + lost

    dx, dx_tol = product(vocab, g, g_tol, w64, w.dtype, x.dtype == F32)
    x64 = torch.where(there, x64, 0.0)
    dw = [product(tokens, a.t().contiguous(), t.t().contiguous(), b, x.dtype, grad_dtype == F32)
          for a, t, b in zip(g.view(workers, tokens, vocab), g_tol.view(workers, tokens, vocab),
                             x64.view(workers, tokens, cols))]
    return (dx.view(x.shape), dx_tol.view(x.shape), torch.stack([a for a, _ in dw]), torch.stack([t for _, t in dw]))


def close(got, want, tol, dtype, name):
    tol = tol + HALF_STEP[dtype] * (want.abs() + tol) + TINY
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"{name}: {float((off / tol).max())} of the tolerance"


SIZES = [(1, 1, 1, 1), (1, 1, 2, 8), (1, 3, 100, 7), (2, 5, 127, 64), (1, 64, 128, 65), (3, 33, 129, 63), (1, 255, 255, 96),
         (1, 256, 256, 256), (2, 129, 257, 200), (1, 257, 511, 72), (3, 100, 1000, 515), (1, 300, 5003, 48),
         (8, 37, 777, 264), (1, 1, 3001, 768), (1, 17, 2048, 1032), (2, 520, 300, 128)]


@pytest.mark.parametrize("workers,tokens,vocab,cols", SIZES)
@pytest.mark.parametrize("x_dtype", [F32, BF16])
@pytest.mark.parametrize("w_dtype", [F32, BF16])
def test_forward(workers, tokens, vocab, cols, x_dtype, w_dtype):
    ids = torch.int32 if tokens % 2 else torch.int64
    x, w, targets, _ = inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, tokens + vocab + cols, ids=ids)
    scale = 0.75 if vocab % 2 else -1.5
    loss, lse = run_forward(x, w, targets, scale)
    want = losses_in_64(*logits_in_64(x, w, scale), targets, vocab)
    close(lse.flatten(), want[0], want[1], F32, "lse")
    close(loss.flatten(), want[2], want[3], F32, "loss")
    assert bool((loss.flatten()[~want[4]] == 0).all())


@pytest.mark.parametrize("workers,tokens,vocab,cols", SIZES)
@pytest.mark.parametrize("x_dtype", [F32, BF16])
@pytest.mark.parametrize("w_dtype", [F32, BF16])
@pytest.mark.parametrize("grad_dtype", [F32, BF16])
def test_backward(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype):
    ids = torch.int64 if tokens % 2 else torch.int32
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, tokens * vocab + cols, ids=ids)
    scale = -1.25 if vocab % 2 else 1.0
    lse = torch.logsumexp(logits_in_64(x, w, scale)[0], 1).float().view(workers, tokens)
    dx, dw = run_backward(x, w, targets, scale, lse, dloss, grad_dtype)
    want = gradients_in_64(x, w, targets, scale, lse, dloss, grad_dtype)
    close(dx, want[0], want[1], x_dtype, "dx")
    close(dw, want[2], want[3], grad_dtype, "dw")
    padded = (targets < 0) | (targets >= vocab)
    assert bool((dx[padded] == 0).all())


@pytest.mark.parametrize("x_dtype", [F32, BF16])
@pytest.mark.parametrize("grad_dtype", [F32, BF16])
def test_some_outputs_only_and_adding(x_dtype, grad_dtype):
    x, w, targets, dloss = inputs(2, 140, 700, 136, x_dtype, BF16, 9)
    _, lse = run_forward(x, w, targets, 1.0)
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    assert same_bits(run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, want=(True, False))[0], dx)
    assert same_bits(run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, want=(False, True))[1], dw)
    start = torch.randn(dw.shape, generator=gen(3)).to(grad_dtype).to(DEV)
    _, added = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, start=start)
    exact, tol = gradients_in_64(x, w, targets, 1.0, lse, dloss, grad_dtype)[2:]
    close(added, exact + start.double(), tol + U * (exact.abs() + start.double().abs()), grad_dtype, "dw")
    # with fp32 sums the addition is one rounding
    if grad_dtype == F32:
        assert same_bits(added, dw + start)


def test_forward_in_pieces():
    """Weights that are laid out for the tiles a piece at a time, and many rows, whose maxima and sums are
    joined a piece at a time."""
    for tokens, vocab, cols, x_dtype, w_dtype in [(40, 50257, 1030, BF16, F32), (65536, 33000, 8, BF16, BF16)]:
        x, w, targets, _ = inputs(1, tokens, vocab, cols, x_dtype, w_dtype, 21)
        loss, lse = run_forward(x, w, targets, 1.0)
        at = torch.arange(0, tokens, max(tokens // 500, 1), device=DEV)
        want = losses_in_64(*logits_in_64(x[:, at], w, 1.0), targets[:, at], vocab)
        close(lse[0, at], want[0], want[1], F32, "lse")
        close(loss[0, at], want[2], want[3], F32, "loss")


@pytest.mark.parametrize("x_dtype,w_dtype,grad_dtype", [(BF16, BF16, F32), (F32, BF16, BF16), (BF16, F32, BF16)])
def test_backward_in_pieces(x_dtype, w_dtype, grad_dtype):
    workers, tokens, vocab, cols = 2, 8192, 9001 if w_dtype == BF16 else 18000, 24
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, 22)
    _, lse = run_forward(x, w, targets, 1.0)
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    want = gradients_in_64(x, w, targets, 1.0, lse, dloss, grad_dtype)
    close(dx, want[0], want[1], x_dtype, "dx")
    close(dw, want[2], want[3], grad_dtype, "dw")


def test_padded_tokens_hold_anything():
    """NaN and infinities at tokens without a target reach nothing but their own lse."""
    x, w, targets, dloss = inputs(2, 150, 400, 80, BF16, BF16, 31, pad=False)
    bad = torch.zeros(2, 150, dtype=torch.bool, device=DEV)
    bad[0, 3], bad[0, 149], bad[1, 0], bad[1, 70] = True, True, True, True
    targets[bad] = -1
    clean = x.clone()
    x[0, 3], x[0, 149], x[1, 0], x[1, 70] = float("nan"), float("inf"), -float("inf"), 3e38
    dloss[0, 3], dloss[1, 0] = float("nan"), float("inf")
    loss, lse = run_forward(x, w, targets, 1.0)
    want_loss, want_lse = run_forward(clean, w, targets, 1.0)
    assert same_bits(loss, want_loss) and same_bits(lse[~bad], want_lse[~bad])
    assert bool((loss[bad] == 0).all())
    for grad_dtype in (F32, BF16):
        dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
        good = torch.where(bad, 0.0, dloss)
        want_dx, want_dw = run_backward(clean, w, targets, 1.0, want_lse, good, grad_dtype)
        assert same_bits(dw, want_dw) and same_bits(dx, want_dx)
        assert bool((dx[bad] == 0).all())


def test_a_batch_without_any_target():
    x, w, targets, dloss = inputs(3, 40, 300, 64, BF16, BF16, 33, pad=False)
    targets[1] = -1
    loss, lse = run_forward(x, w, targets, 1.0)
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, F32)
    assert bool((loss[1] == 0).all()) and bool((dx[1] == 0).all()) and bool((dw[1] == 0).all())
    assert bool((dw[0] != 0).any()) and bool((dw[2] != 0).any())


def test_nan_and_infinity_stay_in_their_row():
    x, w, targets, dloss = inputs(1, 90, 300, 64, F32, F32, 34, pad=False)
    x[0, 5, 7], x[0, 70, 0] = float("nan"), float("inf")
    loss, _ = run_forward(x, w, targets, 1.0)
    assert bool(loss[0, [5, 70]].isnan().all())
    keep = torch.ones(90, dtype=torch.bool, device=DEV)
    keep[[5, 70]] = False
    assert bool(loss[0, keep].isfinite().all())


def test_far_logits():
    """Rows whose logits lie at +-1000, all alike, or with one far above the others: maxima are subtracted."""
    vocab, cols = 1000, 8
    w = torch.zeros(vocab, cols)
    w[:, 0], w[17, 1], w[:, 2] = 1.0, 1.0, torch.linspace(-1, 1, vocab).bfloat16().float()
    x = torch.zeros(1, 6, cols)
    x[0, 0, 0], x[0, 1, 0], x[0, 2, 1], x[0, 3, 1], x[0, 4, 2] = 1000.0, -1000.0, 200.0, -200.0, 512.0
    targets = torch.tensor([[3, 999, 17, 17, 0, 500]])
    x, w, targets = x.to(DEV), w.to(DEV), targets.to(DEV)
    for dtype in (F32, BF16):
        a, b = x.to(dtype), w.to(dtype)
        loss, lse = run_forward(a, b, targets, 1.0)
        want = losses_in_64(*logits_in_64(a, b, 1.0), targets, vocab)
        close(lse[0], want[0], want[1], F32, "lse")
        close(loss[0], want[2], want[3], F32, "loss")
        dloss = torch.ones(1, 6, device=DEV)
        dx, dw = run_backward(a, b, targets, 1.0, lse, dloss, F32)
        wanted = gradients_in_64(a, b, targets, 1.0, lse, dloss, F32)
        close(dx, wanted[0], wanted[1], dtype, "dx")
        close(dw, wanted[2], wanted[3], F32, "dw")


def test_masked_vocabulary():
    """Rows of the weight that send their logits to minus infinity count as absent."""
    x, w, targets, dloss = inputs(1, 50, 520, 64, BF16, BF16, 35, pad=False)
    x[..., 0] = 1.0
    w[:, 0] = 0.0
    targets.clamp_(max=200)
    kept = run_forward(x, w[:256].contiguous(), targets, 1.0)
    w[256:] = 0.0
    w[256:, 0] = -float("inf")
    got = run_forward(x, w, targets, 1.0)
    for a, b in zip(got, kept):
        assert bool(a.isfinite().all())
        assert bool(((a - b).abs() <= 16 * U * (1 + b.abs())).all())


@pytest.mark.parametrize("workers,tokens,vocab,cols", [(2, 50, 520, 64), (3, 100, 1000, 515), (2, 40, 300, 6144),
                                                       (1, 2100, 9000, 264)])
@pytest.mark.parametrize("x_dtype", [F32, BF16])
@pytest.mark.parametrize("w_dtype", [F32, BF16])
def test_masked_vocabulary_of_every_type(workers, tokens, vocab, cols, x_dtype, w_dtype):
    """A logit of minus infinity counts as nothing whatever the operands' types, whether an entry of the weight is
    infinite or a product passes fp32's range; and a token that holds an infinity is no number, but no other is."""
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, 36)
    x[..., 0] = x[..., 0].abs() + 0.25
    x[:, ::3, 0], x[..., 1] = 1.0, 1.1e30
    w[:, :2] = 0.0
    kind = torch.arange(vocab, device=DEV) % 5
    keep = kind < 3
    w[kind == 3] = 0.0
    w[kind == 3, 0] = -math.inf
    w[kind == 4, 1] = -1.3e30
    w[9::10, 1] = -1.303e30  # whose second plane is of the other sign
    inside = (targets >= 0) & (targets < vocab)
    targets = torch.where(inside, targets // 5 * 5, targets)
    loss, lse = run_forward(x, w, targets, 1.0)
    rest = torch.where(inside, targets // 5 * 3, targets)  # among the entries that count
    rest[rest >= vocab] = -1
    kept = w[keep].contiguous()
    want = losses_in_64(*logits_in_64(x, kept, 1.0), rest, int(keep.sum()))
    close(lse.flatten(), want[0], want[1], F32, "lse")
    close(loss.flatten(), want[2], want[3], F32, "loss")
    for grad_dtype in (F32, BF16):
        dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
        want = gradients_in_64(x, kept, rest, 1.0, lse, dloss, grad_dtype)
        # nought times infinity in the column that holds them
        close(dx[..., 1:], want[0][..., 1:], want[1][..., 1:], x_dtype, "dx")
        assert bool((dw[:, ~keep] == 0).all())
        close(dw[:, keep], want[2], want[3], grad_dtype, "dw")
    x[0, 7] = math.inf
    _, again = run_forward(x, w, targets, 1.0)
    others = torch.ones(workers, tokens, dtype=torch.bool, device=DEV)
    others[0, 7] = False
    assert same_bits(again[others], lse[others]) and bool(again[~others].isnan().all())
    targets[0, 7] = 0
    dx_bad, dw_bad = run_backward(x, w, targets, 1.0, again, dloss, BF16)
    assert same_bits(dx_bad[others], dx[others]) and bool(dx_bad[~others].isnan().all())
    assert same_bits(dw_bad[1:], dw[1:]) and bool(dw_bad[0].isnan().all())


def test_backward_is_the_forwards_by_differences():
    """Central differences of a weighted sum of the losses along one direction of x and w, in 64 bits, against
    the kernel's gradients."""
    workers, tokens, vocab, cols, scale, step = 2, 30, 400, 72, 0.5, 1e-4
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, F32, F32, 41)
    dirs = [torch.randn(t.shape, generator=gen(42 + i), dtype=torch.float64).to(DEV) for i, t in enumerate((x, w))]
    _, lse = run_forward(x, w, targets, scale)
    dx, dw = run_backward(x, w, targets, scale, lse, dloss, F32)
    there = (targets >= 0) & (targets < vocab)
    at = torch.where(there, targets, 0).long()

    def total(t):
        a, b = x.double() + t * dirs[0], w.double() + t * dirs[1]
        l = scale * (a.flatten(0, 1) @ b.t().contiguous()).view(workers, tokens, vocab)
        loss = torch.logsumexp(l, -1) - l.gather(-1, at[..., None])[..., 0]
        return float((loss * there * dloss.double()).sum())

    by_difference = (total(step) - total(-step)) / (2 * step)
    by_gradient = float((dx.double() * dirs[0]).sum() + (dw.double().sum(0) * dirs[1]).sum())
    # step^2 of the third derivative (logits move by about 10 a unit), and the products' 2^-16 of their sizes
    size = float((dx.double() * dirs[0]).abs().sum() + (dw.double() * dirs[1]).abs().sum())
    assert abs(by_difference - by_gradient) < 60 * 1000 * step ** 2 + 3 * 2.0 ** -16 * size


def test_replays_and_streams_give_the_same_bits():
    workers, tokens, vocab, cols = 2, 200, 900, 130
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, BF16, F32, 50)
    loss, lse, dx = torch.empty_like(dloss), torch.empty_like(dloss), torch.empty_like(x)
    dw = torch.empty(workers, vocab, cols, device=DEV)
    ws = sm.bytes_tensor(sm.signmuon_linear_cross_entropy_workspace_bytes(workers * tokens, vocab, cols, BF16, F32), DEV)
    back = sm.bytes_tensor(sm.signmuon_linear_cross_entropy_backward_workspace_bytes(workers, tokens, vocab, cols, BF16,
                                                                                    F32, F32), DEV)

    def refresh(i):
        for t, new in zip((x, w, targets, dloss), inputs(workers, tokens, vocab, cols, BF16, F32, 60 + 7 * i)):
            t.copy_(new)

    def call(stream=None):
        sm.signmuon_linear_cross_entropy(x, w, targets, 1.0, loss, lse, ws, stream=stream)
        sm.signmuon_linear_cross_entropy_backward(x, w, targets, 1.0, lse, dloss, dx, dw, back, stream=stream)

    outs = [loss, lse, dx, dw]
    replays_like_eager(call, outs, refresh)
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    call(torch.cuda.Stream())
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert same_bits(a, b)


WALKS = [(2, 1100, 9000, 200), (1, 4096, 20000, 520), (4, 512, 12000, 264), (1, 3000, 2500, 1030)]


@pytest.mark.parametrize("workers,tokens,vocab,cols", WALKS)
@pytest.mark.parametrize("x_dtype,w_dtype,grad_dtype", [(BF16, BF16, BF16), (BF16, BF16, F32), (BF16, F32, F32),
                                                        (F32, F32, F32), (F32, BF16, BF16)])
def test_workgroups_that_walk_several_tiles(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype):
    """More tiles than run at once, of several slices: the loads of the next tile, and the stores of the one
    before, are under way during a tile."""
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, 71)
    loss, lse = run_forward(x, w, targets, 1.0)
    want = losses_in_64(*logits_in_64(x, w, 1.0), targets, vocab)
    close(lse.flatten(), want[0], want[1], F32, "lse")
    close(loss.flatten(), want[2], want[3], F32, "loss")
    del want
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    want = gradients_in_64(x, w, targets, 1.0, lse, dloss, grad_dtype)
    close(dx, want[0], want[1], x_dtype, "dx")
    close(dw, want[2], want[3], grad_dtype, "dw")
    again = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    assert same_bits(again[0], dx) and same_bits(again[1], dw)
    start = torch.randn(dw.shape, generator=gen(3)).to(grad_dtype).to(DEV)
    _, added = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, start=start)
    close(added, want[2] + start.double(), want[3] + U * (want[2].abs() + start.double().abs()), grad_dtype, "dw")


# (of one tile of 128 x 128 or a few, with hundreds of slices of k; rows that are no whole vectors)
LONG = [(1, 1, 130, 8200), (2, 3, 257, 5000), (1, 129, 200, 4099), (3, 200, 333, 6152)]


@pytest.mark.parametrize("workers,tokens,vocab,cols", LONG)
@pytest.mark.parametrize("x_dtype,w_dtype,grad_dtype", [(BF16, BF16, BF16), (BF16, BF16, F32), (BF16, F32, F32),
                                                        (F32, F32, F32), (F32, BF16, BF16)])
def test_logits_of_long_rows(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype):
    """Few logits of many columns, whose sums come in parts."""
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, 83)
    loss, lse = run_forward(x, w, targets, 1.0)
    want = losses_in_64(*logits_in_64(x, w, 1.0), targets, vocab)
    close(lse.flatten(), want[0], want[1], F32, "lse")
    close(loss.flatten(), want[2], want[3], F32, "loss")
    assert bool((loss.flatten()[~want[4]] == 0).all())
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    want = gradients_in_64(x, w, targets, 1.0, lse, dloss, grad_dtype)
    close(dx, want[0], want[1], x_dtype, "dx")
    close(dw, want[2], want[3], grad_dtype, "dw")
    again = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    assert same_bits(again[0], dx) and same_bits(again[1], dw)
    start = torch.randn(dw.shape, generator=gen(3)).to(grad_dtype).to(DEV)
    _, added = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, start=start)
    close(added, want[2] + start.double(), want[3] + U * (want[2].abs() + start.double().abs()), grad_dtype, "dw")


@pytest.mark.parametrize("workers,tokens,vocab,cols", [(8, 1000, 65, 44), (1, 5000, 256, 384), (3, 2100, 130, 330)])
@pytest.mark.parametrize("x_dtype,w_dtype,grad_dtype", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, F32, F32),
                                                        (F32, BF16, BF16)])
def test_small_vocabularies(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype):
    """Few entries of dw, whose sums over many tokens come in parts."""
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, 91)
    lse = torch.logsumexp(logits_in_64(x, w, 1.0)[0], 1).float().view(workers, tokens)
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    want = gradients_in_64(x, w, targets, 1.0, lse, dloss, grad_dtype)
    close(dx, want[0], want[1], x_dtype, "dx")
    close(dw, want[2], want[3], grad_dtype, "dw")
    again = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    assert same_bits(again[0], dx) and same_bits(again[1], dw)
    start = torch.randn(dw.shape, generator=gen(3)).to(grad_dtype).to(DEV)
    _, added = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, start=start)
    close(added, want[2] + start.double(), want[3] + U * (want[2].abs() + start.double().abs()), grad_dtype, "dw")
    if grad_dtype == F32:  # one rounding
        assert same_bits(added, dw + start)


@pytest.mark.parametrize("x_dtype,w_dtype,grad_dtype,vocab", [(BF16, BF16, F32, 4500), (F32, BF16, BF16, 4500),
                                                              (BF16, F32, BF16, 9000)])
def test_pieces_of_many_tokens(x_dtype, w_dtype, grad_dtype, vocab):
    """g of two pieces of the vocabulary, of two workers."""
    x, w, targets, dloss = inputs(2, 32768, vocab, 24, x_dtype, w_dtype, 92)
    _, lse = run_forward(x, w, targets, 1.0)
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    want = gradients_in_64(x, w, targets, 1.0, lse, dloss, grad_dtype)
    close(dx, want[0], want[1], x_dtype, "dx")
    close(dw, want[2], want[3], grad_dtype, "dw")
    start = torch.randn(dw.shape, generator=gen(3)).to(grad_dtype).to(DEV)
    _, added = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, start=start)
    close(added, want[2] + start.double(), want[3] + U * (want[2].abs() + start.double().abs()), grad_dtype, "dw")


@pytest.mark.parametrize("tokens,vocab,cols", [(1500, 6000, 1304), (2048, 4000, 2048), (300, 130, 264), (7000, 300, 48)])
@pytest.mark.parametrize("x_dtype,grad_dtype", [(BF16, F32), (F32, BF16), (BF16, BF16), (F32, F32)])
def test_one_gradient_alone(tokens, vocab, cols, x_dtype, grad_dtype):
    """At sizes of each tile. Where x and dw are of one type, what is asked for changes no bits of it."""
    x, w, targets, dloss = inputs(1, tokens, vocab, cols, x_dtype, BF16, 93)
    _, lse = run_forward(x, w, targets, 1.0)
    dx = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, want=(True, False))[0]
    dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, want=(False, True))[1]
    want = gradients_in_64(x, w, targets, 1.0, lse, dloss, grad_dtype)
    close(dx, want[0], want[1], x_dtype, "dx")
    close(dw, want[2], want[3], grad_dtype, "dw")
    both = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    assert same_bits(both[1], dw) and (x_dtype != grad_dtype or same_bits(both[0], dx))


def test_long_rows_of_padding_and_masked_vocabulary():
    """In parts of k too: tokens without a target hold anything, and a vocabulary entry of minus infinity in
    BF16 counts as nothing."""
    x, w, targets, dloss = inputs(2, 40, 300, 6144, BF16, BF16, 84)
    x, w = x.abs(), w.clone()
    w[17] = -math.inf
    targets[targets == 17] = 18
    targets[1, 3:] = -100
    x[1, 3:] = math.nan
    loss, lse = run_forward(x, w, targets, 1.0)
    l, l_tol = logits_in_64(x.nan_to_num(), w[torch.arange(300, device=DEV) != 17], 1.0)
    there = ((targets >= 0) & (targets < 300)).flatten()
    rest = torch.where(targets > 17, targets - 1, targets)
    want = losses_in_64(l, l_tol, torch.where(there.view(2, 40), rest, -1), 299)
    # nought times infinity is no number: of tokens that hold a nought, nor is that logit
    nought = (x == 0).any(-1).flatten() & there
    assert int(nought.sum()) == 1
    assert bool(lse.flatten()[nought].isnan().all()) and bool(loss.flatten()[nought].isnan().all())
    counts = there & ~nought
    close(lse.flatten()[counts], want[0][counts], want[1][counts], F32, "lse")
    close(loss.flatten()[~nought], want[2][~nought], want[3][~nought], F32, "loss")
    w[17] = 0
    lse = torch.where(counts.view(2, 40), lse, 0)
    dx, dw = run_backward(x, w, targets, 1.0, torch.where(there.view(2, 40), lse, math.nan), dloss, BF16)
    want = gradients_in_64(x.nan_to_num(), w, targets, 1.0, lse, dloss, BF16)
    close(dx, want[0], want[1], BF16, "dx")
    close(dw, want[2], want[3], BF16, "dw")


@pytest.mark.parametrize("workers,tokens,vocab,cols", [(1, 1, 900, 256), (1, 5, 2000, 130), (8, 2, 700, 264), (1, 128, 5000, 96),
                                                       (3, 42, 300, 4100)])
@pytest.mark.parametrize("x_dtype,w_dtype,grad_dtype", [(BF16, BF16, BF16), (BF16, F32, BF16), (F32, BF16, BF16),
                                                        (BF16, BF16, F32)])
def test_few_tokens_keep_g_whole(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype):
    """Up to 128 tokens, BF16 results are off by their own rounding, and by no rounding of g."""
    x, w, targets, dloss = inputs(workers, tokens, vocab, cols, x_dtype, w_dtype, 85, pad=tokens > 1)
    _, lse = run_forward(x, w, targets, 1.0)
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
    want = gradients_in_64(x, w, targets, 1.0, lse, dloss, grad_dtype, whole_g=True)
    close(dx, want[0], want[1], x_dtype, "dx")
    close(dw, want[2], want[3], grad_dtype, "dw")
    start = torch.randn(dw.shape, generator=gen(3)).to(grad_dtype).to(DEV)
    _, added = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype, start=start)
    close(added, want[2] + start.double(), want[3] + U * (want[2].abs() + start.double().abs()), grad_dtype, "dw")


def test_more_than_2_31_entries_of_x():
    """Rows of x and dx at offsets past 2^31 entries; dw sums 2^21 tokens."""
    tokens, vocab, cols = 1 << 21, 64, 1032
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(1, tokens, cols, generator=g, device=DEV, dtype=BF16)
    w = (torch.randn(vocab, cols, generator=g, device=DEV) * (2 / math.sqrt(cols))).to(BF16)
    targets = torch.randint(-2, vocab, (1, tokens), generator=g, device=DEV)
    dloss = torch.randn(1, tokens, generator=g, device=DEV)
    loss, lse = run_forward(x, w, targets, 1.0)
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, F32)
    total = torch.zeros(1, vocab, cols, dtype=torch.float64, device=DEV)
    total_tol = torch.zeros_like(total)
    for t0 in range(0, tokens, 1 << 17):
        part = slice(t0, t0 + (1 << 17))
        args = x[:, part], w, targets[:, part], 1.0, lse[:, part], dloss[:, part], F32
        want = gradients_in_64(*args)
        close(dx[:, part], want[0], want[1], BF16, "dx")
        total += want[2]
        total_tol += want[3] + 4 * math.sqrt(tokens) * U * want[2].abs().amax()
        losses = losses_in_64(*logits_in_64(x[:, part], w, 1.0), targets[:, part], vocab)
        close(loss[0, part], losses[2], losses[3], F32, "loss")
    close(dw, total, total_tol, F32, "dw")


def test_more_than_2_31_entries_of_dw():
    workers, tokens, vocab, cols = 2, 3, 1 << 20, 2040
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(workers, tokens, cols, generator=g, device=DEV, dtype=BF16)
    w = torch.randn(vocab, cols, generator=g, device=DEV, dtype=BF16).mul_(0.05)
    targets = torch.tensor([[0, vocab - 1, 524288], [-1, 77, vocab - 2]], device=DEV)
    dloss = torch.ones(workers, tokens, device=DEV)
    loss, lse = run_forward(x, w, targets, 1.0)
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, BF16)
    l, l_tol = logits_in_64(x, w, 1.0)
    losses = losses_in_64(l, l_tol, targets, vocab)
    close(loss.flatten(), losses[2], losses[3], F32, "loss")
    rows = torch.cat([torch.arange(0, vocab, 9973, device=DEV), torch.tensor([0, 77, 524288, vocab - 2, vocab - 1], device=DEV)])
    p = torch.exp(l - lse.double().flatten()[:, None]).view(workers, tokens, vocab)
    for m in range(workers):
        one = (rows[None, :] == targets[m][:, None]).double()
        gr = torch.where((targets[m] >= 0)[:, None], p[m][:, rows] - one, 0.0)
        want = gr.t() @ x[m].double()
        # g in one plane, and a sum of three products; exponentials of logits that are off by l_tol
        size = gr.abs().t() @ x[m].double().abs()
        tol = (2.0 ** -8 + 8 * U) * size + (p[m][:, rows] * (l_tol.view(workers, tokens, vocab)[m][:, rows] + 60 * U)).t() @ x[m].double().abs()
        close(dw[m, rows], want, tol, BF16, "dw")
