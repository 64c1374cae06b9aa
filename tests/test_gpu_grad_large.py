"""The gradient operators where offsets pass 2^31 elements and 2^32 bytes: parts
of the results at both ends of the buffers against 64 bits, and every row that
has to be zero."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, TINY
from test_gpu_f8 import E4, E5, quantised, same_values, tolerance
from test_gpu_layer_norm import U, backward_in_64, statistics

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name_the_case(request):
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def random(shape, dtype, seed):
    return torch.randn(shape, dtype=dtype, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))


def near(got, want, tol):
    tol = tol + HALF_STEP[got.dtype] * (want.abs() + tol) + TINY
    assert bool(((got.cpu().double() - want).abs() <= tol).all())


def test_a_table_and_tokens_of_many_rows():
    vocab, cols, tokens = 1 << 20, 2047, 1100003
    table = random((vocab, cols), torch.float32, 1)
    ids = torch.randint(0, vocab, (tokens,), device=DEV)
    ids[0], ids[-1], ids[-2] = 0, vocab - 1, vocab
    y = torch.empty(tokens, cols, dtype=torch.bfloat16, device=DEV)
    assert y.numel() > 2 ** 31
    sm.signmuon_embedding(ids, table, 1.0, y)
    for at in range(0, tokens, 100000):
        rows = ids[at:at + 100000]
        want = table[rows.clamp(max=vocab - 1)].bfloat16()
        want[rows == vocab] = 0
        assert torch.equal(y[at:at + 100000], want)


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("add", [False, True])
def test_a_stack_of_large_gradients(grad_dtype, add):
    workers, vocab, cols, tokens = 3, 1 << 20, 1001, 700
    ids = torch.randint(0, vocab, (workers, tokens), device=DEV)
    ids[:, 0], ids[:, 1], ids[:, 2:40], ids[:, 40] = vocab - 1, 0, 12345, -1
    dy = random((workers, tokens, cols), torch.float32, 2)
    grad = torch.full((workers, vocab, cols), 1.0 if add else float("nan"), dtype=grad_dtype, device=DEV)
    assert grad.numel() > 2 ** 31
    ws = sm.bytes_tensor(sm.signmuon_embedding_workspace_bytes(workers, tokens, vocab, cols), DEV)
    sm.signmuon_embedding_backward(ids, dy, 1.0, grad, ws, accumulate=add)
    for m in range(workers):
        there, place = ids[m][ids[m] >= 0].unique(return_inverse=True)
        terms = dy[m][ids[m] >= 0].cpu().double()
        zeros = torch.zeros(len(there), cols, dtype=torch.float64)
        want, size = (zeros.index_add(0, place.cpu(), v) for v in (terms, terms.abs()))
        want = want + (1.0 if add else 0.0)
        near(grad[m][there], want, 1.001 * 40 * U * size + U * want.abs())
        rest = torch.ones(vocab, dtype=torch.bool, device=DEV)
        rest[there] = False
        for at in range(0, vocab, 1 << 17):
            rows = grad[m, at:at + (1 << 17)]
            wrong = (rows != (1.0 if add else 0.0)).any(-1)
            assert not bool((wrong & rest[at:at + (1 << 17)]).any())


@pytest.mark.parametrize("rows,cols", [(1100002, 1025), (34002, 32773)])
def test_layer_norm_of_many_rows(rows, cols):
    workers, eps = 2, float(torch.tensor(1e-5))
    x, dy = random((workers * rows, cols), torch.bfloat16, 3), random((workers * rows, cols), torch.bfloat16, 4)
    assert x.numel() > 2 ** 31
    gamma, beta = 1 + 0.1 * random((cols,), torch.float32, 5), random((cols,), torch.float32, 6)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(workers * rows, device=DEV) for _ in range(2))
    dgamma, dbeta = (torch.empty(workers, cols, device=DEV) for _ in range(2))
    ws = sm.bytes_tensor(sm.signmuon_layer_norm_workspace_bytes(workers, rows, cols), DEV)
    sm.signmuon_layer_norm(x, gamma, beta, eps, y, mean, rstd)
    sm.signmuon_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, workers=workers)
    for part in (slice(0, 20), slice(rows - 10, rows + 10), slice(workers * rows - 20, workers * rows)):
        px, pm, pr = x[part].cpu(), mean[part].cpu(), rstd[part].cpu()
        m, m_tol, r, r_tol = statistics(px, eps)
        assert bool(((pm.double() - m).abs() <= m_tol + TINY).all())
        assert bool(((pr.double() - r).abs() <= r_tol).all())
        g = gamma.cpu().double()
        scaled = (px.double() - m[:, None]) * r[:, None] * g
        want = scaled + beta.cpu().double()
        tol = m_tol[:, None] * (r[:, None] * g).abs() + scaled.abs() * ((r_tol / r)[:, None] + 3 * U) + U * want.abs()
        near(y[part], want, 1.01 * tol)
        want = backward_in_64(dy[part].cpu(), px, gamma.cpu(), pm, pr, 1)
        near(dx[part], want[0], 1.01 * want[1])
    step = max(1, (1 << 25) // cols)
    for w in range(workers):
        sums = [torch.zeros(cols, dtype=torch.float64, device=DEV) for _ in range(4)]
        for at in range(w * rows, (w + 1) * rows, step):
            part = slice(at, min(at + step, (w + 1) * rows))
            d = dy[part].double()
            t = d * ((x[part].double() - mean[part].double()[:, None]) * rstd[part].double()[:, None])
            for s, v in zip(sums, (t, t.abs(), d, d.abs())):
                s += v.sum(0)
        # roundings of random sign along a chain of at most every row add as its root, each of u times a partial
        # sum; the partial sums are below the sizes' sum
        for got, want, size in ((dgamma, *sums[:2]), (dbeta, *sums[2:])):
            assert bool(((got[w].double() - want).abs() <= U * (rows ** 0.5 + 30) * size).all())


@pytest.mark.parametrize("fmt", [E4, E5])
def test_operands_of_many_rows(fmt):
    rows, cols = 2200005, 1000
    x = random((rows, cols), torch.bfloat16, 7)
    assert x.numel() > 2 ** 31
    q, qs = sm.f8_empty((rows, cols), fmt, DEV)
    t, ts = sm.f8_empty((cols, rows), fmt, DEV)
    sm.signmuon_f8_quant(x, q, qs, t, ts)
    begin = rows // 128 * 128 - 256
    for part in (slice(0, 256), slice(begin, rows)):
        want, scale = quantised(x[part].cpu(), fmt)
        assert torch.equal(qs[part].cpu(), scale) and same_values(q[part].cpu(), want)
    tail = x[begin:].cpu().t().contiguous()
    want, scale = quantised(tail, fmt)
    assert same_values(t[:, begin:].cpu(), want)
    assert torch.equal(ts[:, begin // 128:begin // 128 + 3].cpu(), scale[:, :3])


@pytest.mark.parametrize("batch,m,n,k", [(1, 2200005, 1030, 1024), (1, 2200005, 1032, 1024), (2, 1100001, 1000, 1100)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_products_of_many_rows(batch, m, n, k, out_dtype):
    a, b = sm.f8_empty((batch, m, k), E4, DEV), sm.f8_empty((batch, n, k), E5, DEV)
    sm.signmuon_f8_quant(random((batch, m, k), torch.bfloat16, 8), *a)
    sm.signmuon_f8_quant(random((batch, n, k), torch.bfloat16, 9), *b)
    out = torch.full((batch, m, n), float("nan"), dtype=out_dtype, device=DEV)
    assert a[0].numel() > 2 ** 31 and out.numel() > 2 ** 31
    ws = sm.bytes_tensor(sm.signmuon_f8_matmul_workspace_bytes(batch, m, n, k), DEV)
    sm.signmuon_f8_matmul(*a, *b, k, out, ws)
    for i in range(batch):
        for part in (slice(0, 33), slice(m // 2, m // 2 + 20), slice(m - 33, m)):
            pairs = []
            for q, s in ((a[0][i, part], a[1][i, part]), (b[0][i], b[1][i])):
                q, s = q.cpu(), s.cpu()
                blocks = torch.exp2(s[:, :q.shape[-1] // 128].double() - 127)
                pairs.append((q, s, (q.double().unflatten(-1, (-1, 128)) * blocks.unsqueeze(-1)).flatten(-2), blocks))
            near(out[i, part], pairs[0][2] @ pairs[1][2].t(), tolerance(out_dtype, *pairs, E4, E5))
        for at in range(0, m, 200000):
            assert bool(out[i, at:at + 200000].isfinite().all())
