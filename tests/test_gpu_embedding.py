"""Embedding lookup and its gradient against a plain implementation in 64
bits. Tolerances count roundings: a sum of n fp32 terms is off by at most
n * 2^-24 times the sum of their sizes, scaling and adding by 2^-24 of the
value each, storage by half a step of its type."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, TINY, Guarded, replays_like_eager, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name_the_case(request):
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make_ids(kind, workers, tokens, vocab, dtype, seed):
    g = gen(seed)
    if kind == "words":  # frequency falls as one over the rank
        u = torch.rand(workers, tokens, generator=g, dtype=torch.float64)
        ids = (float(vocab + 1) ** u).long().sub(1).clamp(0, vocab - 1)
    elif kind == "one":
        ids = torch.full((workers, tokens), vocab - 1, dtype=torch.long)
    elif kind == "distinct":
        ids = torch.stack([torch.randperm(max(vocab, tokens), generator=g)[:tokens] % vocab for _ in range(workers)])
    elif kind == "padding":
        ids = torch.full((workers, tokens), -1, dtype=torch.long)
    else:  # some outside the table, on both sides, far away too
        ids = torch.randint(0, vocab, (workers, tokens), generator=g)
        far = [-1, vocab, -2 ** 31, 2 ** 31 - 1] + ([-2 ** 63, 2 ** 62, 2 ** 32] if dtype == torch.int64 else [])
        where = torch.rand(workers, tokens, generator=g) < 0.4
        ids[where] = torch.tensor(far)[torch.randint(0, len(far), (int(where.sum()),), generator=g)]
    return ids.to(dtype)


@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (5, 3, 2), (64, 100, 64), (65, 300, 63), (257, 1000, 96),
                                               (1000, 257, 515), (33, 50, 768), (7, 20, 1025), (130, 40, 4099)])
@pytest.mark.parametrize("table_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
def test_lookup(tokens, vocab, cols, table_dtype, y_dtype):
    dtype = torch.int32 if tokens % 2 else torch.int64
    ids = make_ids("some", 1, tokens, vocab, dtype, tokens)[0]
    table = torch.randn(vocab, cols, generator=gen(1)).to(table_dtype)
    scale = 27.7
    out = Guarded((tokens, cols), y_dtype)
    sm.signmuon_embedding(ids.to(DEV), table.to(DEV), scale, out.t)
    torch.cuda.synchronize()
    out.check("y")
    there = (ids >= 0) & (ids < vocab)
    scale32 = float(torch.tensor(scale, dtype=torch.float32))
    want = torch.where(there[:, None], table.double()[ids.long().clamp(0, vocab - 1)] * scale32, 0.0)
    tol = (2.0 ** -24 + HALF_STEP[y_dtype] * (1 + 2.0 ** -24)) * want.abs() + TINY
    assert bool(((out.t.cpu().double() - want).abs() <= tol).all())


def test_lookup_keeps_nan_and_infinity_of_the_table_out_of_padding():
    table = torch.tensor([[float("nan"), float("inf"), -float("inf"), 1.0]], device=DEV)
    ids = torch.tensor([[0, -1], [1, 0]], device=DEV)
    y = torch.empty(2, 2, 4, device=DEV)
    sm.signmuon_embedding(ids, table, 2.0, y)
    y = y.cpu()
    assert torch.equal(y[0, 1], torch.zeros(4)) and torch.equal(y[1, 0], torch.zeros(4))
    assert torch.equal(torch.nan_to_num(y[0, 0], nan=5.0, posinf=6.0, neginf=7.0), torch.tensor([5.0, 6.0, 7.0, 2.0]))


def gradient_in_64(ids, dy, scale, vocab):
    """(gradient, sum of sizes, terms) of each row."""
    w, t, c = dy.shape
    grad = torch.zeros(w, vocab + 1, c, dtype=torch.float64)
    size = torch.zeros_like(grad)
    count = torch.zeros(w, vocab + 1, dtype=torch.float64)
    ids = ids.long()
    ids = torch.where((ids >= 0) & (ids < vocab), ids, vocab)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    for m in range(w):
        grad[m].index_add_(0, ids[m], dy[m].double() * scale)
        size[m].index_add_(0, ids[m], (dy[m].double() * scale).abs())
        count[m].index_add_(0, ids[m], torch.ones(t, dtype=torch.float64))
    return grad[:, :-1], size[:, :-1], count[:, :-1]


def workspace(workers, tokens, vocab, cols):
    return Guarded((sm.signmuon_embedding_workspace_bytes(workers, tokens, vocab, cols),), torch.uint8)


def check_gradient(kind, workers, tokens, vocab, cols, id_dtype, dy_dtype, grad_dtype, add, scale=1.7, seed=3):
    ids = make_ids(kind, workers, tokens, vocab, id_dtype, seed)
    dy = torch.randn(workers, tokens, cols, generator=gen(seed + 1)).to(dy_dtype)
    grad = Guarded((workers, vocab, cols), grad_dtype)
    old = torch.randn(workers, vocab, cols, generator=gen(seed + 2)).to(grad_dtype)
    if add:
        grad.t.copy_(old)
    ws = workspace(workers, tokens, vocab, cols)
    sm.signmuon_embedding_backward(ids.to(DEV), dy.to(DEV), scale, grad.t, ws.t, accumulate=add)
    torch.cuda.synchronize()
    grad.check("grad")
    ws.check("workspace")
    want, size, count = gradient_in_64(ids, dy, scale, vocab)
    tol = 1.001 * (count[..., None] + 1) * 2.0 ** -24 * size
    if add:
        want = want + old.double()
        tol = tol + 2.0 ** -24 * want.abs()
    tol = tol + HALF_STEP[grad_dtype] * (want.abs() + tol) + TINY
    got = grad.t.cpu()
    assert bool(((got.double() - want).abs() <= tol).all())
    untouched = (count == 0)[..., None].expand_as(want)
    if add:
        assert same_bits(got[untouched], old[untouched])
    else:
        assert bool((got[untouched] == 0).all())


SIZES = [(1, 1, 1, 1), (1, 1, 70000, 5), (1, 15, 40, 256), (2, 16, 257, 257), (1, 17, 3, 64), (3, 63, 64, 3),
         (2, 65, 65, 769), (1, 129, 1000, 1024), (1, 4095, 256, 31), (2, 4096, 300, 40), (1, 4097, 5003, 33),
         (3, 8193, 2000, 20), (1, 20001, 70001, 9)]


@pytest.mark.parametrize("kind", ["words", "one", "distinct", "padding", "some"])
@pytest.mark.parametrize("workers,tokens,vocab,cols", SIZES)
def test_gradient(kind, workers, tokens, vocab, cols):
    odd = (tokens + len(kind)) % 2
    check_gradient(kind, workers, tokens, vocab, cols, torch.int64 if odd else torch.int32, torch.float32,
                   torch.float32, False)


@pytest.mark.parametrize("dy_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("kind,workers,tokens,vocab,cols", [("words", 2, 700, 500, 515), ("one", 1, 5000, 7, 130),
                                                            ("some", 3, 300, 1000, 768)])
def test_gradient_types(dy_dtype, grad_dtype, add, kind, workers, tokens, vocab, cols):
    check_gradient(kind, workers, tokens, vocab, cols, torch.int64, dy_dtype, grad_dtype, add)


def test_gradient_is_the_lookups():
    """<dy, d lookup> = <gradient, d table>: by differences of the (linear) lookup."""
    vocab, tokens, cols = 50, 300, 96
    ids = make_ids("some", 1, tokens, vocab, torch.int64, 9).to(DEV)
    dy = torch.randn(1, tokens, cols, generator=gen(10)).to(DEV)
    table, change = (torch.randn(vocab, cols, generator=gen(s)).to(DEV) for s in (11, 12))
    y = [torch.empty(1, tokens, cols, device=DEV) for _ in range(2)]
    sm.signmuon_embedding(ids, table, 1.5, y[0])
    sm.signmuon_embedding(ids, table + change, 1.5, y[1])
    grad = torch.empty(1, vocab, cols, device=DEV)
    sm.signmuon_embedding_backward(ids, dy, 1.5, grad, workspace(1, tokens, vocab, cols).t)
    by_difference = (dy.double() * (y[1].double() - y[0].double())).sum()
    by_gradient = (grad.double() * change.double()).sum()
    # each y and each table entry is off by 2^-24 of sizes up to about 10, over 300 * 96 terms of random sign
    assert abs(float(by_difference - by_gradient)) < 300 * 96 * 10 * 2.0 ** -23


def test_two_runs_and_two_streams_give_the_same_bits():
    ids = make_ids("words", 3, 6000, 900, torch.int64, 5).to(DEV)
    dy = torch.randn(3, 6000, 200, generator=gen(6)).to(DEV)
    outs = [torch.full((3, 900, 200), 9.0, device=DEV) for _ in range(3)]
    spaces = [workspace(3, 6000, 900, 200).t for _ in range(3)]
    streams = [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for o, w, s in zip(outs, spaces, streams):  # two of them at once, on other streams
        sm.signmuon_embedding_backward(ids, dy, 1.0, o, w, stream=s)
    torch.cuda.synchronize()
    assert same_bits(outs[0], outs[1]) and same_bits(outs[0], outs[2])


def test_a_captured_gradient_replays_like_eager_calls():
    workers, tokens, vocab, cols = 2, 5000, 700, 130
    ids = torch.empty(workers, tokens, dtype=torch.int64, device=DEV)
    dy = torch.empty(workers, tokens, cols, device=DEV)
    y = torch.empty(workers, tokens, cols, device=DEV)
    table = torch.randn(vocab, cols, generator=gen(8)).to(DEV)
    grad = torch.empty(workers, vocab, cols, device=DEV)
    ws = workspace(workers, tokens, vocab, cols)

    def refresh(i):
        ids.copy_(make_ids(["words", "one", "some"][i], workers, tokens, vocab, torch.int64, i))
        dy.copy_(torch.randn(workers, tokens, cols, generator=gen(20 + i)))

    def call():
        sm.signmuon_embedding(ids, table, 2.0, y)
        sm.signmuon_embedding_backward(ids, dy, 2.0, grad, ws.t)

    replays_like_eager(call, [y, grad], refresh)


@pytest.mark.parametrize("cols", [1, 3, 4, 5, 255, 256, 257, 258, 259, 260, 513, 515, 769, 1025, 1027])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
def test_adding_to_columns_at_the_border_of_two_waves(cols, grad_dtype):
    """Each column is added to once, whatever part of it shares a vector with the
    columns of another wave; rows of one segment and rows that several share."""
    for kind, tokens, vocab in (("some", 3000, 4000), ("words", 3000, 4000), ("one", 500, 3)):
        check_gradient(kind, 3, tokens, vocab, cols, torch.int32, torch.bfloat16, grad_dtype, True)
