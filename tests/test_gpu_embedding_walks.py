"""The table's gradient where its waves go round their loops more than once (more
than 16 sorted tokens a wave, more than 64), and where rows without a token are
written beside the sums (more than 96 MB of gradient), with groups of rows that
hundreds of tokens share, that no token has, and that all have one.

The terms are whole numbers and the scale a power of two, so that every sum is
exact in fp32 in any order: results are compared bit for bit, and one token left
out or added twice shows."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, Guarded, embed_segment, same_bits

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _name_the_case(request):
    if request.node.get_closest_marker("gpu") is None:
        yield
        return
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def make_ids(kind, workers, tokens, vocab, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if kind == "words":  # frequency falls as one over the rank
        u = torch.rand(workers, tokens, generator=g, device=DEV, dtype=torch.float64)
        return (float(vocab + 1) ** u).long().sub(1).clamp(0, vocab - 1)
    if kind == "one":  # one id in every place, among the first rows
        return torch.full((workers, tokens), min(5, vocab - 1), device=DEV)
    if kind == "distinct":
        return torch.stack([torch.randperm(max(vocab, tokens), generator=g, device=DEV)[:tokens] % vocab
                            for _ in range(workers)])
    if kind == "row by row":  # whole groups of rows have tokens, and those behind them have none
        return torch.arange(tokens, device=DEV).expand(workers, tokens) % vocab
    if kind == "pairs":  # each id twice or thrice, many rows ending in one wave
        return torch.randint(0, min(vocab, max(1, tokens // 2)), (workers, tokens), generator=g, device=DEV)
    ids = torch.randint(0, vocab, (workers, tokens), generator=g, device=DEV)  # padding in three of ten places
    return torch.where(torch.rand(workers, tokens, generator=g, device=DEV) < 0.3, -1, ids)


def row_sums(ids, dy, vocab):
    """Sums of the rows with each id, in 64 bits: differences of running sums of whole numbers (adding at an index
    takes its turns one by one where many have the same)."""
    want = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=DEV)
    if len(ids):
        ids, order = ids.sort(stable=True)
        rows, counts = ids.unique_consecutive(return_counts=True)
        ends = dy[order].double().t().contiguous().cumsum(1)[:, counts.cumsum(0) - 1]
        want[rows] = ends.diff(dim=1, prepend=torch.zeros_like(ends[:, :1])).t()
    return want


def check(kind, workers, tokens, vocab, cols, dy_dtype, grad_dtype, add):
    g = torch.Generator(device=DEV).manual_seed(7)
    ids = make_ids(kind, workers, tokens, vocab, 3)
    # at most 8 * 131072 in size: exact in fp32
    dy = torch.randint(-8, 9, (workers, tokens, cols), generator=g, device=DEV).to(dy_dtype)
    grad = Guarded((workers, vocab, cols), grad_dtype)
    old = torch.randint(-100, 101, (workers, vocab, cols), generator=g, device=DEV).to(grad_dtype) if add else None
    if add:
        grad.t.copy_(old)
    ws = Guarded((sm.signmuon_embedding_workspace_bytes(workers, tokens, vocab, cols),), torch.uint8)
    sm.signmuon_embedding_backward(ids, dy, 2.0, grad.t, ws.t, accumulate=add)
    torch.cuda.synchronize()
    grad.check("grad")
    ws.check("workspace")
    there = ids >= 0
    rows = (ids + vocab * torch.arange(workers, device=DEV)[:, None])[there]
    want = row_sums(rows, dy[there], workers * vocab).view(workers, vocab, cols) * 2
    if add:
        want += old
    assert float(want.abs().max()) < 2 ** 24
    # + 0.0: a sum that cancels may be -0 on one side
    assert same_bits(grad.t + 0.0, want.to(F32).to(grad_dtype) + 0.0)


# (workers, tokens, vocab, cols), sorted tokens a wave
LONG = [((8, 16384, 20000, 768), 32), ((8, 8192, 9000, 2048), 32), ((4, 70000, 5003, 300), 64),
        ((8, 16384, 300, 4096), 128), ((2, 131072, 70001, 515), 64), ((1, 16000, 40, 20000), 128),
        ((3, 50001, 1000, 4099), 256)]
KINDS = ["words", "one", "distinct", "row by row", "pairs", "padding"]


@pytest.mark.parametrize("sizes,seg", LONG)
def test_segments(sizes, seg):
    workers, tokens, _, cols = sizes
    assert embed_segment(workers, tokens, cols) == seg


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [s for s, _ in LONG])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("add", [False, True])
def test_long_segments(sizes, kind, add):
    odd = (len(kind) + sizes[3]) % 2
    check(kind, *sizes, BF16 if odd else F32, F32, add)


@pytest.mark.gpu
@pytest.mark.parametrize("dy_dtype", [F32, BF16])
@pytest.mark.parametrize("kind", KINDS)
def test_long_segments_to_bf16(dy_dtype, kind):
    check(kind, 8, 16384, 300, 1030, dy_dtype, BF16, False)
    check(kind, 8, 16384, 300, 1030, dy_dtype, BF16, True)


# more than 96 MB: rows of a group that one workgroup fills with zeros (12 KB, at most 32 rows)
WIDE = [((1, 4096, 50000, 768), F32), ((1, 20000, 50257, 768), F32), ((2, 5000, 60001, 1025), BF16),
        ((8, 5000, 200003, 33), F32), ((8, 20000, 150000, 64), BF16), ((255, 300, 9999, 17), F32),
        ((3, 1, 130001, 96), F32)]


@pytest.mark.parametrize("sizes,grad_dtype", WIDE)
def test_sizes_of_wide_gradients(sizes, grad_dtype):
    workers, _, vocab, cols = sizes
    assert workers * vocab * cols * (2 if grad_dtype == BF16 else 4) > 96 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,grad_dtype", WIDE)
@pytest.mark.parametrize("kind", KINDS)
def test_zeros_beside_the_sums(sizes, grad_dtype, kind):
    check(kind, *sizes, BF16 if len(kind) % 2 else F32, grad_dtype, False)
