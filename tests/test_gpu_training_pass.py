"""The operators together, as a training step uses them: token ids to rows of
the table, layer norm, an 8-bit product with its two gradients, the norm's and
the table's gradients, all of them stacks [Mw][R][C] that signmuon_step reads,
and the weights that it updates read by the next pass.

Each stage is compared with the 64-bit result of that stage's own inputs as they
lie in GPU memory, with the tolerances of the operators' own tests; the step is
compared with the oracle on the same stacks."""
import numpy as np
import pytest
import torch

import oracle
import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, TINY, replays_like_eager
from test_gpu_embedding import gradient_in_64
from test_gpu_f8 import E4, E5, quantised, same_values, tolerance
from test_gpu_layer_norm import backward_in_64, statistics

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS, BETA, ETA = float(torch.tensor(1e-5)), 0.9, 1e-3


@pytest.fixture(autouse=True)
def _name_the_case(request):
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()


class Pass:
    """Buffers of a model of one table, one norm and one product, and the pass
    over `workers` x `tokens` ids, which leaves the four gradients in self.mats.
    The table serves twice: its second use adds to the gradient of the first."""

    def __init__(self, workers, tokens, vocab, cols, inner, act, ns_iters, seed=0):
        g = torch.Generator().manual_seed(seed)
        new = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
        self.sizes = workers, tokens, vocab, cols, inner
        self.act, self.scale = act, cols ** 0.5
        self.start = [0.05 * torch.randn(vocab, cols, generator=g), 0.1 * torch.randn(inner, cols, generator=g),
                      1 + 0.1 * torch.randn(1, cols, generator=g), 0.1 * torch.randn(1, cols, generator=g)]
        self.mats = [sm.Matrix(grad=new((workers,) + tuple(w.shape)), momentum=new((workers,) + tuple(w.shape)),
                               packed=new((workers, sm.signmuon_packed_words(w.numel())), torch.int64),
                               weight=new(w.shape), polar_out=new((workers,) + tuple(w.shape)),
                               vote_out=new(w.shape, torch.int8)) for w in self.start]
        self.params = sm.Params(workers=workers, beta=BETA, eta=ETA, ns_iters=ns_iters)
        self.step_space = sm.workspace_tensor(self.mats, self.params, DEV)
        self.ids = torch.zeros((workers, tokens), dtype=torch.int32, device=DEV)
        self.ids2 = torch.zeros((workers, tokens), dtype=torch.int64, device=DEV)
        self.dz, self.d2 = new((workers, tokens, inner), act), new((workers, tokens, cols), act)
        self.x, self.y, self.dy, self.dx = (new((workers, tokens, cols), act) for _ in range(4))
        self.z = new((workers, tokens, inner), act)
        self.mean, self.rstd = new((workers, tokens)), new((workers, tokens))
        self.yq, self.yt = sm.f8_empty((workers, tokens, cols), E4, DEV), sm.f8_empty((workers, cols, tokens), E4, DEV)
        self.wq, self.wt = sm.f8_empty((inner, cols), E4, DEV), sm.f8_empty((cols, inner), E4, DEV)
        self.dq, self.dt = (sm.f8_empty((workers, tokens, inner), E5, DEV),
                            sm.f8_empty((workers, inner, tokens), E5, DEV))
        need = [sm.signmuon_embedding_workspace_bytes(workers, tokens, vocab, cols),
                sm.signmuon_layer_norm_workspace_bytes(workers, tokens, cols),
                sm.signmuon_f8_matmul_workspace_bytes(workers, tokens, inner, cols),
                sm.signmuon_f8_matmul_workspace_bytes(workers, tokens, cols, inner),
                sm.signmuon_f8_matmul_workspace_bytes(workers, inner, cols, tokens)]
        self.space = sm.bytes_tensor(max(need), DEV)  # one after the other on one stream: one workspace

    def reset(self):
        for m, w in zip(self.mats, self.start):
            m.weight.copy_(w)
            m.momentum.zero_()

    def feed(self, seed):
        workers, tokens, vocab, cols, inner = self.sizes
        g = torch.Generator().manual_seed(seed)
        ids = torch.randint(0, vocab, (2, workers, tokens), generator=g)
        ids[:, :, tokens // 2:] = ids[:, :, tokens // 2:] % 7  # frequent words
        ids[:, 0, tokens - 3:] = -1  # a padded row
        self.ids.copy_(ids[0])
        self.ids2.copy_(ids[1])
        self.dz.copy_(torch.randn(workers, tokens, inner, generator=g) * 1e-3)
        self.d2.copy_(torch.randn(workers, tokens, cols, generator=g) * 1e-2)

    def forward(self):
        table, w, gamma, beta = (m.weight for m in self.mats)
        cols = self.sizes[3]
        sm.signmuon_embedding(self.ids, table, self.scale, self.x)
        sm.signmuon_layer_norm(self.x, gamma.view(-1), beta.view(-1), EPS, self.y, self.mean, self.rstd)
        sm.signmuon_f8_quant(self.y, *self.yq, *self.yt)
        sm.signmuon_f8_quant(w, *self.wq, *self.wt)
        sm.signmuon_f8_matmul(*self.yq, *self.wq, cols, self.z, self.space)

    def backward(self):
        workers, tokens, _, _, inner = self.sizes
        table, w, gamma, beta = self.mats
        sm.signmuon_f8_quant(self.dz, *self.dq, *self.dt)
        sm.signmuon_f8_matmul(*self.dq, *self.wt, inner, self.dy, self.space)
        sm.signmuon_f8_matmul(*self.dt, *self.yt, tokens, w.grad, self.space)
        sm.signmuon_layer_norm_backward(self.dy, self.x, gamma.weight.view(-1), self.mean, self.rstd, self.dx,
                                        gamma.grad, beta.grad, self.space, workers=workers)
        sm.signmuon_embedding_backward(self.ids, self.dx, self.scale, table.grad, self.space)
        sm.signmuon_embedding_backward(self.ids2, self.d2, 1.0, table.grad, self.space, accumulate=True)

    def step(self):
        sm.signmuon_step(self.mats, self.params, self.step_space)

    def run(self):
        self.forward()
        self.backward()
        self.step()


def near(got, want, tol):
    tol = tol + HALF_STEP[got.dtype] * (want.abs() + tol) + TINY
    assert bool(((got.cpu().double() - want).abs() <= tol).all())


def with_values(pair, k):
    """A quantised pair as test_gpu_f8's operands: bytes, scales, values, block scales, on the CPU."""
    q, s = (t.cpu() for t in pair)
    blocks = torch.exp2(s[..., :q.shape[-1] // 128].double() - 127)
    return q, s, (q.double().unflatten(-1, (-1, 128)) * blocks.unsqueeze(-1)).flatten(-2), blocks


def check_quant(pair, x, fmt):
    q, s = quantised(x, fmt)
    assert torch.equal(pair[1].cpu(), s) and same_values(pair[0].cpu(), q)


def check_product(out, a, b, k, fa, fb):
    a, b = with_values(a, k), with_values(b, k)
    if b[0].dim() < a[0].dim():
        b = tuple(t.expand((a[0].shape[0],) + t.shape) for t in b)
    near(out, a[2] @ b[2].transpose(-1, -2), tolerance(out.dtype, a, b, fa, fb))


def check_gradients(p):
    workers, tokens, vocab, cols, inner = p.sizes
    table, w, gamma, beta = (m.weight.cpu() for m in p.mats)
    scale = float(torch.tensor(p.scale, dtype=torch.float32))
    ids, x, y = p.ids.cpu().long(), p.x.cpu(), p.y.cpu()
    want = torch.where((ids >= 0)[..., None], table.double()[ids.clamp(min=0)] * scale, 0.0)
    near(p.x, want, U * want.abs())
    flat = x.view(-1, cols)
    mean, mean_tol, rstd, rstd_tol = (t.view(workers, tokens) for t in statistics(flat, EPS))
    assert bool(((p.mean.cpu().double() - mean).abs() <= 1.01 * mean_tol + U * mean.abs() + TINY).all())
    assert bool(((p.rstd.cpu().double() - rstd).abs() <= 1.01 * rstd_tol + U * rstd).all())
    # y from the statistics: the difference is off by the mean's error and u of itself, times rstd, gamma, plus beta
    d = x.double() - mean[..., None]
    t = d * rstd[..., None] * gamma.double()
    tol = (gamma.double().abs() * (rstd[..., None] * mean_tol[..., None] + d.abs() * rstd_tol[..., None]) +
           6 * U * (t.abs() + beta.double().abs()))
    near(p.y, t + beta.double(), 1.01 * tol)
    check_quant(p.yq, y, E4)
    check_quant(p.yt, y.transpose(1, 2), E4)
    check_quant(p.wq, w, E4)
    check_quant(p.wt, w.t(), E4)
    check_quant(p.dq, p.dz.cpu(), E5)
    check_quant(p.dt, p.dz.cpu().transpose(1, 2), E5)
    check_product(p.z, p.yq, p.wq, cols, E4, E4)
    check_product(p.dy, p.dq, p.wt, inner, E5, E4)
    check_product(p.mats[1].grad, p.dt, p.yt, tokens, E5, E4)
    want = backward_in_64(p.dy.cpu().view(-1, cols), flat, gamma.view(-1), p.mean.cpu().view(-1),
                          p.rstd.cpu().view(-1), workers)
    for got, v, tol in zip((p.dx.view(-1, cols), p.mats[2].grad.view(workers, cols), p.mats[3].grad.view(workers, cols)),
                           want[::2], want[1::2]):
        near(got, v, 1.01 * tol)
    first = gradient_in_64(ids, p.dx.cpu(), p.scale, vocab)
    second = gradient_in_64(p.ids2.cpu(), p.d2.cpu(), 1.0, vocab)
    # the first is stored in fp32 and the second's sum added to it
    tol = sum(1.001 * (count[..., None] + 1) * U * size for _, size, count in (first, second)) + U * first[0].abs()
    near(p.mats[0].grad, first[0] + second[0], 1.001 * tol + U * (first[0] + second[0]).abs())


def check_step(p, before, ns_iters):
    for m, (momentum, weight) in zip(p.mats, before):
        m_ref, w_ref = momentum.copy(), weight.copy()
        _, _, u_ref = oracle.step_matrix(m.grad.cpu().numpy(), m_ref, w_ref, BETA, ETA, ns_iters, oracle.F32, want_u=True)
        u = m.polar_out.cpu().numpy()
        assert np.array_equal(m.momentum.cpu().numpy(), m_ref)
        assert np.linalg.norm(u.astype(np.float64) - u_ref) <= 1e-5 * np.linalg.norm(u_ref)
        packed = m.packed.cpu().numpy().view(np.uint64)
        for i in range(u.shape[0]):
            assert np.array_equal(oracle.sign_pack(u[i]), packed[i])
        w = weight.copy()
        assert np.array_equal(m.vote_out.cpu().numpy(), oracle.vote_update(packed, w, ETA))
        assert np.array_equal(m.weight.cpu().numpy(), w)


SIZES = [(2, 300, 517, 200, 130), (3, 5, 40, 64, 9), (1, 70, 33, 129, 300)]


@pytest.mark.parametrize("workers,tokens,vocab,cols,inner", SIZES)
@pytest.mark.parametrize("act", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ns_iters", [0, 1])
def test_two_training_steps(workers, tokens, vocab, cols, inner, act, ns_iters):
    p = Pass(workers, tokens, vocab, cols, inner, act, ns_iters)
    p.reset()
    for i in range(2):
        p.feed(10 + i)
        before = [(m.momentum.cpu().numpy(), m.weight.cpu().numpy()) for m in p.mats]
        p.forward()
        p.backward()
        check_gradients(p)
        p.step()
        check_step(p, before, ns_iters)


@pytest.mark.parametrize("act", [torch.float32, torch.bfloat16])
def test_a_captured_step_replays_like_the_eager_one(act):
    p = Pass(2, 300, 517, 200, 130, act, 1)

    def refresh(i):
        p.reset()
        p.feed(20 + i)

    outputs = [p.x, p.y, p.z, p.dy, p.dx]
    for m in p.mats:
        outputs += [m.grad, m.momentum, m.packed, m.weight, m.vote_out]
    replays_like_eager(p.run, outputs, refresh)


def test_two_passes_on_two_streams():
    """Two models at once, each with its own buffers and workspaces."""
    passes = [Pass(2, 300, 517, 200, 130, torch.bfloat16, 1, seed=s) for s in (1, 2)]
    want = []
    for i, p in enumerate(passes):
        p.reset()
        p.feed(30 + i)
        p.run()
        torch.cuda.synchronize()
        want.append([t.clone() for m in p.mats for t in (m.grad, m.weight)])
        p.reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in passes]
    for p, s in zip(passes, streams):
        with torch.cuda.stream(s):
            p.run()
    torch.cuda.synchronize()
    for p, w in zip(passes, want):
        for got, v in zip((t for m in p.mats for t in (m.grad, m.weight)), w):
            assert torch.equal(got, v)
