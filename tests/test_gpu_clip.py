"""The norm of each worker's gradients and clipping by it, against a plain
implementation in 64 bits.

Tolerances: squares and their sum are fp64, so a norm is off by its rounding to
fp32 (u = 2^-24) and far less; a factor is rounded once (u), and so is a product
(half a step of its type)."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, Guarded, replays_like_eager, same_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
UNIT = 16384  # entries that a workgroup takes


@pytest.fixture(autouse=True)
def _name_the_case(request):
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def gradients(workers, counts, dtypes, seed):
    """Tensors whose sizes differ from worker to worker."""
    out = []
    for i, n in enumerate(counts):
        size = torch.exp(2 * torch.randn(workers, 1, generator=gen(seed + 1000 + i)))
        out.append((torch.randn(workers, n, generator=gen(seed + i)) * size).to(dtypes[i % len(dtypes)]))
    return out


def norms_in_64(grads):
    return torch.stack([g.double().square().sum(1) for g in grads]).sum(0).sqrt()


def clip(grads, most):
    """(norms, clipped) from guarded buffers."""
    workers = grads[0].shape[0]
    outs = [Guarded(tuple(g.shape), g.dtype) for g in grads]
    given = [g.to(DEV) for g in grads]
    handle = sm.Gradients(given, [o.t for o in outs])
    norms = Guarded((workers,), torch.float32)
    ws = Guarded((sm.signmuon_grad_norm_workspace_bytes(handle),), torch.uint8)
    sm.signmuon_clip_grads(handle, most, norms.t, ws.t)
    torch.cuda.synchronize()
    for o in outs + [norms, ws]:
        o.check()
    for g, t in zip(grads, given):
        assert same_bits(g, t.cpu())
    return norms.t, [o.t for o in outs]


def check(grads, most, norms, outs):
    want = norms_in_64(grads)
    assert bool(((norms.cpu().double() - want).abs() <= 1.001 * U * want).all())
    most = float(torch.tensor(most, dtype=torch.float32))
    factor = (most / want).clamp(max=1.0)[:, None]
    for g, o in zip(grads, outs):
        exact = g.double() * factor
        assert bool(((o.cpu().double() - exact).abs() <= (HALF_STEP[g.dtype] + 2 * U) * exact.abs() + 2.0 ** -126).all())
        for m in range(g.shape[0]):
            if want[m] <= most:
                assert same_bits(g[m], o[m].cpu())


COUNTS = [[1], [7], [8], [255, 1], [UNIT], [UNIT - 1, UNIT + 1], [3 * UNIT + 5], [1, 2, 3, 4, 5, 6, 7, 8, 9],
          [100003, 1, 64, 2 * UNIT, 999], [17] * 95, [33] * 96, [65] * 97, [129] * 200]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}of{max(c)}")
@pytest.mark.parametrize("workers", [1, 3, 8])
@pytest.mark.parametrize("dtypes", [(torch.float32,), (torch.bfloat16,), (torch.bfloat16, torch.float32)],
                         ids=["f32", "bf16", "both"])
def test_norms_and_clipping(counts, workers, dtypes):
    grads = gradients(workers, counts, dtypes, len(counts) + workers)
    # some workers pass it and some do not
    most = float(norms_in_64(grads).median()) * (1.0 if workers > 1 else 0.3)
    norms, outs = clip(grads, most)
    check(grads, most, norms, outs)
    handle, alone = sm.Gradients([g.to(DEV) for g in grads]), torch.empty(workers, device=DEV)
    sm.signmuon_grad_norm(handle, alone, sm.bytes_tensor(sm.signmuon_grad_norm_workspace_bytes(handle), DEV))
    assert same_bits(alone, norms)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place(dtype):
    grads = gradients(4, [50001, 3, UNIT], (dtype,), 5)
    most = float(norms_in_64(grads).median())
    norms, outs = clip(grads, most)
    given = [g.to(DEV).view(4, 1, -1) for g in grads]  # [Mw][R][C], as the step's stacks
    handle, alone = sm.Gradients(given), torch.empty(4, device=DEV)
    ws = sm.bytes_tensor(sm.signmuon_grad_norm_workspace_bytes(handle), DEV)
    sm.signmuon_clip_grads(handle, most, alone, ws)
    assert same_bits(alone, norms)
    for g, o in zip(given, outs):
        assert same_bits(g.view(4, -1), o)
    # once more: nothing passes the limit by more than the roundings, and the second pass changes little
    sm.signmuon_clip_grads(handle, most * 1.01, alone, ws)
    for g, o in zip(given, outs):
        assert same_bits(g.view(4, -1), o)


def test_sizes_that_squares_in_fp32_do_not_hold():
    grads = [torch.tensor([[3e38, -3e38, 3e38], [1e-30, 2e-30, 2e-30], [0.0, 0.0, 0.0], [3e-42, 0.0, 4e-42]])]
    norms, outs = clip(grads, 2.5e-30)
    want = norms_in_64(grads)
    # 5.2e38 is past fp32; 5e-42 is subnormal there
    assert float(norms[0]) == float("inf") and float(norms[2]) == 0.0
    assert abs(float(norms[1]) - float(want[1])) <= 1.001 * U * float(want[1])
    assert abs(float(norms[3]) - float(want[3])) <= 2.0 ** -149
    exact = grads[0].double() * (2.5e-30 / want).clamp(max=1.0)[:, None]
    assert bool(((outs[0].cpu().double()[1] - exact[1]).abs() <= 3 * U * exact[1].abs()).all())
    # the factor 4.8e-69 is below fp32: zeros, with their signs
    assert bool((outs[0][0] == 0).all())
    assert same_bits(outs[0].cpu()[2:], grads[0][2:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_finite_entries_are_clipped_by_a_norm_past_fp32(dtype):
    grads = [torch.full((2, 5000), 3e38).to(dtype), torch.tensor([[1.0, -2e38], [1.0, 2.0]]).to(dtype)]
    grads[0][1] = 0.5
    norms, outs = clip(grads, 1e38)
    want = norms_in_64(grads)
    assert float(norms[0]) == float("inf") and float(want[0]) > 2e40 and norms[1].isfinite()
    factor = float(torch.tensor(1e38, dtype=torch.float32)) / want[0]
    for g, o in zip(grads, outs):
        exact = g[0].double() * factor
        assert bool(((o[0].cpu().double() - exact).abs() <= (HALF_STEP[dtype] + 2 * U) * exact.abs()).all())
        assert same_bits(o[1].cpu(), g[1])


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kept", [129, 130, 180, 201, 254, 255])
@pytest.mark.parametrize("value", [131, 171, 177, 213, 255])
def test_products_are_rounded_once(value, kept, sign):
    """Products a little beside the middle of two BF16 values, by less than a step of fp32: rounded to fp32 first they
    would be in the middle. The norm is a power of 2, so that the factor is max_norm's bits."""
    middle = kept * 2 ** 24 + 2 ** 23
    factor = round(middle / value)
    assert 2 ** 23 <= factor < 2 ** 25 and abs(factor * value - middle) <= value // 2 < 2 ** 7
    factor -= factor % 2 if factor >= 2 ** 24 else 0
    grads = torch.zeros(3, 17)
    grads[:, 3], grads[0, 0], grads[1, 16], grads[2, 8] = 2.0 ** 40, sign * value, sign * value, sign * value
    most = factor * 2.0 ** 10
    norms, (out,) = clip([grads.bfloat16()], most)
    assert norms.tolist() == [2.0 ** 40] * 3
    # the exact product is a whole number of 2^-30, of 32 bits: to 8 bits, halves to even
    product, drop = factor * value, (factor * value).bit_length() - 8
    low, high = product >> drop, product & (2 ** drop - 1)
    low += high > 2 ** (drop - 1) or (high == 2 ** (drop - 1) and low % 2)
    want = sign * low * 2.0 ** (drop - 30)
    assert [float(out[0, 0]), float(out[1, 16]), float(out[2, 8])] == [want] * 3


def test_a_worker_that_fails_touches_no_other():
    grads = gradients(5, [1000, 70000], (torch.float32,), 8)
    grads[0][1, 3], grads[1][3, 69999] = float("nan"), float("inf")
    norms, outs = clip(grads, 1.0)
    assert norms[[0, 2, 4]].isfinite().all() and norms[1].isnan() and norms[3] == float("inf")
    keep = [g[[0, 2, 4]] for g in grads]
    check(keep, 1.0, norms[[0, 2, 4]], [o[[0, 2, 4]] for o in outs])
    assert all(bool(o[1].isnan().all()) for o in outs)
    bad = outs[1][3].cpu()
    assert bad[69999].isnan() and bool((bad[:69999] == 0).all()) and bool((outs[0][3] == 0).all())


def test_every_entry_counts():
    """One entry among zeros, at the ends of units and tensors: the norm is its size, exactly."""
    counts = [UNIT + 9, 1, 2 * UNIT, 130]
    for tensor, at in [(0, 0), (0, UNIT - 1), (0, UNIT), (0, UNIT + 8), (1, 0), (2, 2 * UNIT - 1), (3, 129), (3, 0)]:
        grads = [torch.zeros(2, n) for n in counts]
        grads[tensor][1, at] = -8.0
        norms, outs = clip(grads, 2.0)
        assert norms.tolist() == [0.0, 8.0] and float(outs[tensor][1, at]) == -2.0
        assert sum(int((o != 0).sum()) for o in outs) == 1


def test_more_than_2_31_entries():
    """A worker's part at an offset past 2^31 entries."""
    n = (1 << 30) + 11
    g = torch.zeros(3, n, dtype=torch.bfloat16, device=DEV)
    g[0, 0], g[1, 5], g[2, n - 1], g[2, 0] = 1.0, 2.0, 3.0, 4.0
    handle, norms = sm.Gradients([g]), torch.empty(3, device=DEV)
    ws = sm.bytes_tensor(sm.signmuon_grad_norm_workspace_bytes(handle), DEV)
    sm.signmuon_clip_grads(handle, 2.5, norms, ws)
    assert norms.tolist() == [1.0, 2.0, 5.0]
    assert [float(v) for v in (g[0, 0], g[1, 5], g[2, n - 1], g[2, 0])] == [1.0, 2.0, 1.5, 2.0]
    assert int(torch.count_nonzero(g)) == 4


def test_replays_and_streams_give_the_same_bits():
    grads = [g.to(DEV) for g in gradients(3, [40000, 5, UNIT + 1], (torch.float32, torch.bfloat16), 20)]
    outs = [torch.empty_like(g) for g in grads]
    handle, norms = sm.Gradients(grads, outs), torch.empty(3, device=DEV)
    ws = sm.bytes_tensor(sm.signmuon_grad_norm_workspace_bytes(handle), DEV)

    def refresh(i):
        for g, new in zip(grads, gradients(3, [40000, 5, UNIT + 1], (torch.float32, torch.bfloat16), 30 + 7 * i)):
            g.copy_(new)

    def call(stream=None):
        sm.signmuon_clip_grads(handle, 100.0, norms, ws, stream=stream)

    replays_like_eager(call, [norms] + outs, refresh)
    want = [t.clone() for t in [norms] + outs]
    torch.cuda.synchronize()
    call(torch.cuda.Stream())
    torch.cuda.synchronize()
    for a, b in zip([norms] + outs, want):
        assert same_bits(a, b)


def test_two_calls_at_once_with_their_own_workspaces():
    streams, calls = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        grads = gradients(4, [300001, 77], (torch.float32,), 60 + i)
        want = clip(grads, 3.0)
        given = [g.to(DEV) for g in grads]
        handle, norms = sm.Gradients(given), torch.empty(4, device=DEV)
        calls.append((handle, norms, sm.bytes_tensor(sm.signmuon_grad_norm_workspace_bytes(handle), DEV), want))
    torch.cuda.synchronize()
    for s, (handle, norms, ws, _) in zip(streams, calls):
        sm.signmuon_clip_grads(handle, 3.0, norms, ws, stream=s)
    torch.cuda.synchronize()
    for handle, norms, _, (n, outs) in calls:
        assert same_bits(norms, n) and all(same_bits(a, b) for a, b in zip(handle.outs, outs))
