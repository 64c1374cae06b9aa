"""The gradient operators at the largest sizes that the header allows, one
dimension at a time.

Products, lookups and the table's gradient take small whole numbers here, whose
sums are exact in fp32 in any order (and which the 8-bit product does not cut: no
product of whole numbers up to 8 is below 2^-6 of another), so they are compared
bit for bit. Layer norm goes through its own tests' comparison with 64 bits."""
import pytest
import torch

import sign_muon_step_amd as sm
import test_gpu_layer_norm as norms
from gpu_util import announce
from grad_util import DEV, Guarded, f8_plan, same_bits
from test_gpu_embedding_walks import check as check_table
from test_gpu_f8 import E4, E5
from test_gpu_f8_walks import FEW_ROWS, TILES

F32, BF16 = torch.float32, torch.bfloat16
TOKENS, DIM, N, K = 1 << 25, 1 << 20, 1 << 21, 1 << 22


@pytest.fixture(autouse=True)
def _name_the_case(request):
    if request.node.get_closest_marker("gpu") is None:
        yield
        return
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def whole_numbers(batch, rows, k, g):
    """Whole numbers up to 8, each block of 128 of a row times a power of two of its own."""
    x = torch.randint(-8, 9, (batch, rows, k), generator=g, device=DEV, dtype=torch.int8).float()
    e = torch.randint(0, 4, (batch, rows, (k + 127) // 128), generator=g, device=DEV)
    return x.mul_(torch.exp2(e.float()).repeat_interleave(128, -1)[..., :k])


def check_product(batch, m, n, k, fa, fb, out_dtype):
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    x, pairs = [], []
    for rows, fmt in ((m, fa), (n, fb)):
        x.append(whole_numbers(batch, rows, k, g))
        pairs.append(sm.f8_empty((batch, rows, k), fmt, DEV))
        sm.signmuon_f8_quant(x[-1], *pairs[-1])
    out = Guarded((batch, m, n), out_dtype)
    ws = Guarded((sm.signmuon_f8_matmul_workspace_bytes(batch, m, n, k),), torch.uint8)
    sm.signmuon_f8_matmul(*pairs[0], *pairs[1], k, out.t, ws.t if ws.nbytes else None)
    torch.cuda.synchronize()
    out.check("out")
    ws.check("workspace")
    for i in range(batch):
        want = x[0][i].double() @ x[1][i].double().t().contiguous()
        assert float(want.abs().max()) < 2 ** 23
        # + 0.0: a sum that cancels may be -0 on one side
        assert same_bits(out.t[i] + 0.0, want.float().to(out_dtype) + 0.0), f"batch entry {i}"


# each limit with the kernel of few rows and with tiles
LARGEST = [(1, 5, 17, K), (1, 200, 140, K), (1, 3, N, 130), (1, 40, N, 130), (1, TOKENS, 1, 1), (255, 2, 33, 700),
           (255, 130, 70, 200)]


def test_plans_of_the_largest():
    assert [f8_plan(*s).tile == 16 for s in LARGEST] == [True, False, True, False, False, True, False]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", LARGEST + [s for s, *_ in FEW_ROWS + TILES])
@pytest.mark.parametrize("fa,fb", [(E4, E4), (E5, E4)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_products_of_whole_numbers(sizes, fa, fb, out_dtype):
    check_product(*sizes, fa, fb, out_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,vocab,cols", [(TOKENS, DIM, 1), (TOKENS, 1000, 3), (5, 2047, DIM), (4, 1, DIM)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lookups(tokens, vocab, cols, dtype):
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.randint(-1, vocab + 1, (tokens,), generator=g, device=DEV)
    table = torch.randint(-100, 101, (vocab, cols), generator=g, device=DEV, dtype=torch.int8).to(dtype)
    y = Guarded((tokens, cols), dtype)
    sm.signmuon_embedding(ids, table, 2.0, y.t)
    torch.cuda.synchronize()
    y.check("y")
    there = (ids >= 0) & (ids < vocab)
    assert same_bits(y.t, torch.where(there[:, None], table[ids.clamp(0, vocab - 1)] * 2, 0.0).to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("workers,tokens,vocab,cols", [(1, TOKENS, DIM, 1), (255, TOKENS // 255, 300, 2),
                                                       (1, 100, 2047, DIM), (1, 3, 1, DIM), (255, 1, 8, 7)])
@pytest.mark.parametrize("kind", ["words", "one", "pairs", "padding"])
@pytest.mark.parametrize("add", [False, True])
def test_table_gradients(workers, tokens, vocab, cols, kind, add):
    check_table(kind, workers, tokens, vocab, cols, BF16 if add else F32, F32, add)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,dtype", [(TOKENS, 2, F32), (3, DIM, F32), (3, DIM, BF16), (2, DIM - 1, BF16)])
def test_layer_norm(rows, cols, dtype):
    norms.test_forward(rows, cols, dtype, True)
    norms.test_backward(1, rows, cols, dtype, F32)


@pytest.mark.gpu
@pytest.mark.parametrize("workers,rows,cols", [(255, 40, 129), (255, 1, 9000)])
def test_layer_norm_of_many_workers(workers, rows, cols):
    norms.test_backward(workers, rows, cols, BF16, F32)


@pytest.mark.gpu
@pytest.mark.parametrize("workers,rows,cols", [(1, TOKENS, 2), (1, TOKENS - 77, 1), (3, 5000, 768), (8, 1024, 300), (2, 40, 9000),
                                               (255, 100, 129), (1, 70001, 1024), (4, 300, DIM // 4), (1, 3001, 5000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("grad_dtype", [F32, BF16])
def test_layer_norm_sums_of_whole_numbers(workers, rows, cols, dtype, grad_dtype):
    """With means of 0 and reciprocal deviations of 1 (which the backward pass is given), the weight's gradient is the sum
    of dy x: exact in whole numbers, so that one row left out or added twice shows."""
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x, dy = (torch.randint(-8, 9, (workers * rows, cols), generator=g, device=DEV, dtype=torch.int8).to(dtype) for _ in range(2))
    gamma, mean, rstd = torch.ones(cols, device=DEV), torch.zeros(workers * rows, device=DEV), torch.ones(workers * rows, device=DEV)
    dx = Guarded((workers * rows, cols), dtype)
    dgamma, dbeta = Guarded((workers, cols), grad_dtype), Guarded((workers, cols), grad_dtype)
    ws = Guarded((sm.signmuon_layer_norm_workspace_bytes(workers, rows, cols),), torch.uint8)
    sm.signmuon_layer_norm_backward(dy, x, gamma, mean, rstd, dx.t, dgamma.t, dbeta.t, ws.t if ws.nbytes else None,
                                    workers=workers)
    torch.cuda.synchronize()
    for o in (dx, dgamma, dbeta, ws):
        o.check()
    for m in range(workers):
        part = slice(m * rows, (m + 1) * rows)
        for got, want in ((dgamma, (dy[part].double() * x[part].double()).sum(0)), (dbeta, dy[part].double().sum(0))):
            assert float(want.abs().max()) < 2 ** 23
            assert same_bits(got.t[m] + 0.0, want.float().to(grad_dtype) + 0.0), f"worker {m}"


@pytest.mark.gpu
@pytest.mark.parametrize("workers,tokens,vocab,cols", [(1, 40, 9, 515), (3, 5000, 700, 130), (2, 16384, 300, 4096)])
@pytest.mark.parametrize("add", [False, True])
def test_nan_and_infinity_at_padding(workers, tokens, vocab, cols, add):
    """What stands at tokens whose id is outside the table does not reach the gradient."""
    g = torch.Generator(device=DEV).manual_seed(4)
    ids = torch.randint(0, vocab, (workers, tokens), generator=g, device=DEV)
    ids[:, ::3], ids[:, 1::7] = -1, vocab
    ids[-1, tokens // 2:] = 1 << 40
    dy = torch.randint(-8, 9, (workers, tokens, cols), generator=g, device=DEV, dtype=torch.int8).bfloat16()
    away = (ids < 0) | (ids >= vocab)
    grads = []
    for value in (0.0, float("nan"), float("inf")):
        dy[away] = value
        grad = torch.full((workers, vocab, cols), 3.0, device=DEV)
        ws = sm.bytes_tensor(sm.signmuon_embedding_workspace_bytes(workers, tokens, vocab, cols), DEV)
        sm.signmuon_embedding_backward(ids, dy, 0.5, grad, ws, accumulate=add)
        grads.append(grad)
    assert bool(grads[0].isfinite().all())
    assert same_bits(grads[0], grads[1]) and same_bits(grads[0], grads[2])
