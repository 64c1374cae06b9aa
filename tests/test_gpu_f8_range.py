"""8-bit products at the limits that the header states: values at the top of fp32's
range, and small products beside large ones that cancel."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV
from test_gpu_f8 import E4, E5, multiply, quantised

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _name_the_case(request):
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()


def on_gpu(x, fmt):
    q, s = sm.f8_empty(x.shape, fmt, DEV)
    sm.signmuon_f8_quant(x.to(DEV), q, s)
    return q.cpu(), s.cpu()


# the kernel of few rows, tiles of 128, and k in parts
SHAPES = [(5, 20, 200), (40, 70, 640), (64, 64, 8192)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("fmt,below,over", [(E4, 240 * 2.0 ** 120, 250 * 2.0 ** 120), (E5, 28672 * 2.0 ** 113, 31000 * 2.0 ** 113)])
def test_values_at_the_top_of_fp32s_range(m, n, k, fmt, below, over):
    """Finite fp32 values that round to 2^128 in 8 bits: a BF16 result has them, an F32 result counts them as
    infinite, and their neighbours' rows are what they are. The largest value below stays exact in both."""
    x, w = torch.full((m, k), below), torch.full((n, k), 2.0 ** -30)
    x[1], x[3] = over, -over
    assert bool(x.isfinite().all())
    a, b = on_gpu(x, fmt), on_gpu(w, fmt)
    for got, y in ((a, x), (b, w)):
        q, s = quantised(y, fmt)
        assert torch.equal(got[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(got[1], s)
    top = torch.full((m, 1), below, dtype=torch.float64)
    top[1], top[3] = 2.0 ** 128, -2.0 ** 128
    want = (top * 2.0 ** -30 * k).expand(m, n)  # a few bits: every partial sum of equal terms is within 2^-23 a term
    for out_dtype in (F32, BF16):
        got = multiply(a, b, k, (m, n), out_dtype).double()
        if out_dtype == F32:
            assert bool((got[1] == float("inf")).all()) and bool((got[3] == -float("inf")).all())
            fine = torch.arange(m).remainder(2).eq(0) | (torch.arange(m) > 3)
            assert bool(((got - want).abs()[fine] <= 2.0 ** -23 * k * want.abs()[fine]).all())
        else:
            assert bool(((got - want).abs() <= (2.0 ** -23 * k + 2.0 ** -8) * want.abs()).all())


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_small_products_beside_large_ones_that_cancel(m, n, k):
    """1 - 1 from two groups of k and seven products of 2^-15 beside the first: an F32 result is their exact sum; a BF16 one
    may cut each of them (8 * 2^-13 at most), as the header says."""
    x, w = torch.zeros(m, k), torch.ones(n, k)
    x[:, 0], x[:, 1:8], x[:, 128] = 1.0, 2.0 ** -9, -1.0
    w[:, 1:8] = 2.0 ** -6
    a, b = on_gpu(x, E4), on_gpu(w, E4)
    want = 7 * 2.0 ** -15
    assert bool((multiply(a, b, k, (m, n), F32) == want).all())
    got = multiply(a, b, k, (m, n), BF16).double()
    assert bool(((got - want).abs() <= 8 * 2.0 ** -13).all())
