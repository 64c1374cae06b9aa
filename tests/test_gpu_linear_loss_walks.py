"""The loss's matrix products in every tile, with more tiles than run at once and several slices of k, and at the sizes of
whole output layers: the plan that a size is meant for is asserted, and every entry is compared with 64 bits.

Roundings of many terms are taken as independent, so that a slice of k that is left out or taken twice shows: by
Hoeffding's inequality a sum of terms, each off by at most a share e of itself, is off by more than 10 e times the root
of the sum of their squares once in 10^21."""
import math

import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, TINY, loss_grad_plan, loss_plan, same_bits
from test_gpu_linear_loss import U, inputs, logits_in_64, losses_in_64, run_backward, run_forward

F32, BF16 = torch.float32, torch.bfloat16
COMPUTE_UNITS = 256


@pytest.fixture(autouse=True)
def _name_the_case(request):
    if request.node.get_closest_marker("gpu") is None:
        yield
        return
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def size(sizes, x, w, g):
    return sizes, (x, w, g)


# a product, its tile and parts of k: (workers, tokens, vocab, cols), the types of x, w and dw
DX = [((256, 256, 1), [size((1, 6280, 307, 3968), BF16, BF16, BF16), size((1, 6280, 307, 3968), BF16, F32, BF16),
                       size((8, 1024, 520, 4096), BF16, BF16, BF16), size((1, 4289, 305, 5848), BF16, BF16, F32)]),
      ((256, 256, 3), [size((1, 4745, 2649, 1704), BF16, F32, BF16), size((1, 5581, 1812, 1424), BF16, F32, F32),
                       size((2, 2807, 522, 1424), F32, F32, F32)]),
      ((256, 128, 1), [size((8, 990, 451, 2080), BF16, F32, BF16)]),
      ((256, 128, 3), [size((1, 7576, 2644, 544), BF16, F32, BF16)]),
      ((128, 256, 1), [size((8, 618, 633, 3168), BF16, F32, F32)]),
      ((128, 256, 3), [size((1, 867, 2144, 5536), BF16, F32, F32), size((1, 797, 584, 5768), F32, F32, BF16)]),
      ((128, 128, 1), [size((3, 2135, 300, 2320), BF16, BF16, BF16), size((3, 700, 303, 5174), BF16, F32, BF16),
                       size((1, 7581, 308, 2072), BF16, F32, F32), size((1, 4416, 312, 2243), BF16, F32, F32)]),
      ((128, 128, 3), [size((2, 405, 2384, 4684), BF16, F32, BF16), size((1, 659, 1714, 5516), BF16, F32, F32),
                       size((1, 6718, 483, 530), F32, F32, BF16)]),
      ((128, 128, 5), [size((3, 2462, 2985, 269), BF16, F32, F32), size((1, 7640, 1151, 288), F32, F32, F32)])]
LOGITS = [((256, 256, 3), [size((1, 514, 13098, 775), F32, F32, BF16)]),
          ((256, 128, 3), [size((3, 2393, 535, 991), F32, F32, BF16)]),
          ((128, 128, 3), [size((2, 132, 11641, 880), F32, F32, F32)])]
# (of dw, parts of the tokens are for half of the compute units' places: their tiles go round once)
DW = [((256, 256, 4), [size((2, 6721, 6928, 136), BF16, BF16, BF16)]),
      ((256, 256, 5), [size((2, 2305, 182, 6272), F32, F32, BF16)]),
      ((256, 128, 7), [size((1, 14145, 18432, 32), BF16, BF16, BF16)]),
      ((128, 256, 5), [size((2, 3516, 309, 3968), F32, BF16, BF16)]),
      ((128, 256, 1), [size((8, 700, 2300, 1000), BF16, BF16, F32)]),
      ((128, 128, 5), [size((1, 7590, 7561, 287), BF16, BF16, BF16), size((3, 2342, 7287, 72), F32, BF16, BF16),
                       size((2, 2518, 11594, 65), F32, BF16, BF16)])]
CASES = [(name, plan, s, t) for name, table in (("dx", DX), ("logits", LOGITS), ("dw", DW))
         for plan, cases in table for s, t in cases]
# whole output layers: eight workers' batches for the step, with the table in BF16 and in the step's own fp32, and a
# large block's
LAYERS = [((8, 1024, 50257, 768), (BF16, BF16, F32), (256, 256, 5)), ((8, 1024, 50257, 768), (BF16, F32, F32), (256, 256, 8)),
          ((1, 8192, 32000, 4096), (BF16, BF16, BF16), (256, 256, 1))]


def plan_of(product, sizes, types):
    workers, tokens, vocab, cols = sizes
    x, w, g = (sm._ACT[t] for t in types)
    p = loss_grad_plan(*sizes, x, w, g)
    t = getattr(p, product)
    here = min(vocab, p.piece)
    m, n, batch = {"logits": (workers * tokens, here, 1), "dx": (workers * tokens, cols, 1), "dw": (here, cols, workers)}[product]
    places = COMPUTE_UNITS * (2 if t.tm * t.tn == 128 * 128 else 1)
    return (t.tm, t.tn, t.splits), batch * -(-m // t.tm) * -(-n // t.tn) * t.splits / places


@pytest.mark.parametrize("product,plan,sizes,types", CASES)
def test_plan(product, plan, sizes, types):
    got, rounds = plan_of(product, sizes, types)
    assert got == plan and rounds > (0.8 if product == "dw" else 1.2)
    if product == "logits":
        t = loss_plan(sizes[0] * sizes[1], *sizes[2:], *(sm._ACT[t] for t in types[:2])).logits
        assert (t.tm, t.tn, t.splits) == plan


@pytest.mark.parametrize("sizes,types,plan", LAYERS)
def test_plan_of_layers(sizes, types, plan):
    assert plan_of("dx", sizes, types)[0] == plan
    for product in ("logits", "dw"):
        got, rounds = plan_of(product, sizes, types)
        assert got == (256, 256, 1) and rounds > 1.2


def off_by(a, a_tol, b, share, rows):
    """How far a @ b is off where a is by a_tol, each term by `share` of itself, and sums of `rows` terms in fp32."""
    return 1.01 * (a_tol @ b.abs()) + 10 * share * torch.sqrt(a.square() @ b.square()) + \
        4 * math.sqrt(6 * rows + 4) * U * (a.abs() @ b.abs())


def close(got, want, tol, name):
    tol = tol + HALF_STEP[got.dtype] * (want.abs() + tol) + TINY
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"{name}: {float((off / tol).max())} of the tolerance"


def share_of(result, operand):
    """What g and the operand that meets it are rounded to, for a result of a type: three planes, or one and two."""
    g = 2.0 ** -24 if result == F32 else 2.0 ** -8
    return g + (0.0 if operand == BF16 else 3 * 2.0 ** -24 if result == F32 else 2.0 ** -16)


def check(sizes, types, seed, add):
    workers, tokens, vocab, cols = sizes
    x, w, targets, dloss = inputs(*sizes, types[0], types[1], seed)
    loss, lse = run_forward(x, w, targets, 1.0)
    l, l_tol = logits_in_64(x, w, 1.0)
    want = losses_in_64(l, l_tol, targets, vocab)
    close(lse.flatten(), want[0], want[1], "lse")
    close(loss.flatten(), want[2], want[3], "loss")
    dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, types[2])
    again = run_backward(x, w, targets, 1.0, lse, dloss, types[2])
    assert same_bits(again[0], dx) and same_bits(again[1], dw)
    del again

    # g from the kernel's lse: the exponent is off by the logit's error and by roundings in units of log 2
    there, lse64 = want[4][:, None], lse.double().flatten()[:, None]
    d = torch.where(there, dloss.double().flatten()[:, None], 0.0)
    p = torch.exp(l - lse64)
    g_tol = d.abs() * p * (l_tol + 3 * U * lse64.abs() + 2 * U * l.abs() + 3 * U)
    del l, l_tol
    g = d * p.scatter_add_(1, targets.long().flatten().clamp(0, vocab - 1)[:, None], -there.double())
    del p
    g_tol += 3 * U * g.abs()
    w64, x64 = w.double(), x.double()
    for t0 in range(0, workers * tokens, 2048):  # some rows at a time
        t = slice(t0, t0 + 2048)
        close(dx.flatten(0, 1)[t], g[t] @ w64, off_by(g[t], g_tol[t], w64, share_of(types[0], types[1]), vocab), "dx")
    start = torch.randn(dw.shape, generator=torch.Generator().manual_seed(3)).to(types[2]).to(DEV) if add else None
    added = run_backward(x, w, targets, 1.0, lse, dloss, types[2], start=start)[1] if add else None
    for m in range(workers):
        rows = slice(m * tokens, (m + 1) * tokens)
        a, a_tol = g[rows].t().contiguous(), g_tol[rows].t().contiguous()
        exact = a @ x64[m]
        tol = off_by(a, a_tol, x64[m], share_of(types[2], types[0]), tokens)
        close(dw[m], exact, tol, "dw")
        if add:
            begin = start[m].double()
            close(added[m], exact + begin, tol + U * (exact.abs() + begin.abs()), "dw added to")


@pytest.mark.gpu
@pytest.mark.parametrize("product,plan,sizes,types", CASES)
def test_every_tile(product, plan, sizes, types):
    check(sizes, types, 101, add=product == "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,types,plan", LAYERS)
def test_whole_layers(sizes, types, plan):
    check(sizes, types, 102, add=sizes[0] == 1)


@pytest.mark.gpu
def test_a_vocabulary_of_2_20():
    """dx sums over 2^20 entries, its left operand's rows are 4 MB apart; g of few tokens is met in three planes."""
    workers, tokens, vocab, cols = 2, 3, 1 << 20, 2040
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(workers, tokens, cols, generator=g, device=DEV, dtype=BF16)
    w = torch.randn(vocab, cols, generator=g, device=DEV, dtype=BF16).mul_(0.05)
    targets = torch.tensor([[0, vocab - 1, 524288], [-1, 77, vocab - 2]], device=DEV)
    dloss = torch.tensor([[1.0, -2.0, 0.5], [3.0, 0.25, -1.0]], device=DEV)
    loss, lse = run_forward(x, w, targets, 1.0)
    l, l_tol = logits_in_64(x, w, 1.0)
    want = losses_in_64(l, l_tol, targets, vocab)
    close(lse.flatten(), want[0], want[1], "lse")
    close(loss.flatten(), want[2], want[3], "loss")
    there, lse64 = want[4][:, None], lse.double().flatten()[:, None]
    d = torch.where(there, dloss.double().flatten()[:, None], 0.0)
    p = torch.exp(l - lse64)
    g_tol = d.abs() * p * (l_tol + 3 * U * lse64.abs() + 2 * U * l.abs() + 3 * U)
    exact = d * p.scatter_add_(1, targets.flatten().clamp(0)[:, None], -there.double())
    g_tol += 3 * U * exact.abs()
    for grad_dtype in (BF16, F32):
        dx, dw = run_backward(x, w, targets, 1.0, lse, dloss, grad_dtype)
        assert bool((dx[1, 0] == 0).all())
        for c0 in range(0, cols, 255):
            c = slice(c0, c0 + 255)
            part = w[:, c].double()
            close(dx.flatten(0, 1)[:, c], exact @ part, off_by(exact, g_tol, part, 2.0 ** -24, vocab), "dx")
        rows = torch.cat([torch.arange(0, vocab, 997, device=DEV), torch.tensor([77, 524288, vocab - 2, vocab - 1], device=DEV)])
        for m in range(workers):
            t = slice(m * tokens, (m + 1) * tokens)
            a, a_tol = exact[t][:, rows].t().contiguous(), g_tol[t][:, rows].t().contiguous()
            close(dw[m, rows], a @ x[m].double(), off_by(a, a_tol, x[m].double(), 2.0 ** -24, tokens), "dw")
        del dx, dw
