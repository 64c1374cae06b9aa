"""The operators of a language model's training step together: token ids to rows of
the table, root-mean-square norm straight into an 8-bit product, its output added
to the residual stream and normed again, the loss of an output layer that shares the
table, the gradients of all of it as stacks [Mw][R][C], clipped by each worker's
norm, and the weights that signmuon_step makes of them read by the next pass.

Each stage is compared with the 64-bit result of that stage's own inputs as they lie
in GPU memory, with the tolerances of the operators' own tests; the step is compared
with the oracle on the same stacks."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, TINY, replays_like_eager, same_bits
from test_gpu_clip import check as check_clip
from test_gpu_embedding import gradient_in_64
from test_gpu_f8 import E4, E5
from test_gpu_linear_loss import close, gradients_in_64, logits_in_64, losses_in_64
from test_gpu_rms_norm import backward_in_64, check_f8, normed, stored_sum
from test_gpu_training_pass import check_product, check_quant, check_step, near

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS, BETA, ETA = float(torch.tensor(1e-5)), 0.9, 1e-3
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _name_the_case(request):
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()


class Pass:
    """Buffers of a model of one table, two norms and one product, and the pass over
    `workers` x `tokens` ids and targets, which leaves the four gradients in self.mats."""

    def __init__(self, workers, tokens, vocab, cols, act, ns_iters, most, seed=0):
        g = torch.Generator().manual_seed(seed)
        new = lambda shape, dtype=F32: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
        self.sizes, self.act, self.most = (workers, tokens, vocab, cols), act, most
        self.start = [0.3 * torch.randn(vocab, cols, generator=g), 0.1 * torch.randn(cols, cols, generator=g),
                      1 + 0.1 * torch.randn(1, cols, generator=g), 1 + 0.1 * torch.randn(1, cols, generator=g)]
        self.mats = [sm.Matrix(grad=new((workers,) + tuple(w.shape)), momentum=new((workers,) + tuple(w.shape)),
                               packed=new((workers, sm.signmuon_packed_words(w.numel())), torch.int64),
                               weight=new(w.shape), polar_out=new((workers,) + tuple(w.shape)),
                               vote_out=new(w.shape, torch.int8)) for w in self.start]
        self.params = sm.Params(workers=workers, beta=BETA, eta=ETA, ns_iters=ns_iters)
        self.step_space = sm.workspace_tensor(self.mats, self.params, DEV)
        self.ids, self.targets = (torch.zeros((workers, tokens), dtype=torch.int64, device=DEV) for _ in range(2))
        shape = (workers, tokens, cols)
        self.x, self.y, self.z, self.h, self.y2, self.dy2, self.dh, self.dy, self.dx = (new(shape, act) for _ in range(9))
        self.rstd, self.rstd2, self.loss, self.lse, self.dloss = (new((workers, tokens)) for _ in range(5))
        self.yq, self.yt = sm.f8_empty(shape, E4, DEV), sm.f8_empty((workers, cols, tokens), E4, DEV)
        self.wq, self.wt = sm.f8_empty((cols, cols), E4, DEV), sm.f8_empty((cols, cols), E4, DEV)
        self.dq, self.dt = sm.f8_empty(shape, E5, DEV), sm.f8_empty((workers, cols, tokens), E5, DEV)
        self.table_grad = torch.empty_like(self.mats[0].grad)
        self.norms, self.gradients = new((workers,)), sm.Gradients([m.grad for m in self.mats])
        need = [sm.signmuon_embedding_workspace_bytes(workers, tokens, vocab, cols),
                sm.signmuon_rms_norm_workspace_bytes(workers, tokens, cols),
                sm.signmuon_f8_matmul_workspace_bytes(workers, tokens, cols, cols),
                sm.signmuon_f8_matmul_workspace_bytes(workers, cols, cols, tokens),
                sm.signmuon_linear_cross_entropy_workspace_bytes(workers * tokens, vocab, cols, act, F32),
                sm.signmuon_linear_cross_entropy_backward_workspace_bytes(workers, tokens, vocab, cols, act, F32, F32),
                sm.signmuon_grad_norm_workspace_bytes(self.gradients)]
        self.space = sm.bytes_tensor(max(need), DEV)  # one after the other on one stream: one workspace

    def reset(self):
        for m, w in zip(self.mats, self.start):
            m.weight.copy_(w)
            m.momentum.zero_()

    def feed(self, seed):
        workers, tokens, vocab, _ = self.sizes
        g = torch.Generator().manual_seed(seed)
        ids = torch.randint(0, vocab, (workers, tokens + 1), generator=g)
        ids[:, tokens // 2:] %= 7  # frequent words
        keep = torch.ones(workers, tokens, dtype=torch.bool)
        keep[0, tokens - 2:] = False  # a padded row
        self.ids.copy_(torch.where(keep, ids[:, :-1], -1))
        self.targets.copy_(torch.where(keep, ids[:, 1:], -1))
        self.dloss.copy_(keep / keep.sum(1, keepdim=True).clamp(min=1))

    def forward(self):
        table, w, g1, g2 = (m.weight for m in self.mats)
        cols = self.sizes[3]
        sm.signmuon_embedding(self.ids, table, 1.0, self.x)
        sm.signmuon_rms_norm(self.x, None, g1.view(-1), EPS, y=self.y, q=self.yq[0], q_scale=self.yq[1], rstd=self.rstd)
        sm.signmuon_f8_quant(self.y, None, None, *self.yt)
        sm.signmuon_f8_quant(w, *self.wq, *self.wt)
        sm.signmuon_f8_matmul(*self.yq, *self.wq, cols, self.z, self.space)
        sm.signmuon_rms_norm(self.z, self.x, g2.view(-1), EPS, h=self.h, y=self.y2, rstd=self.rstd2)
        sm.signmuon_linear_cross_entropy(self.y2, table, self.targets, 1.0, self.loss, self.lse, self.space)

    def backward(self):
        workers, tokens, _, cols = self.sizes
        table, w, g1, g2 = self.mats
        sm.signmuon_linear_cross_entropy_backward(self.y2, table.weight, self.targets, 1.0, self.lse, self.dloss, self.dy2,
                                                  table.grad, self.space)
        self.table_grad.copy_(table.grad)
        sm.signmuon_rms_norm_backward(self.dy2, None, self.h, g2.weight.view(-1), self.rstd2, self.dh, g2.grad, self.space,
                                      workers=workers)
        sm.signmuon_f8_quant(self.dh, *self.dq, *self.dt)
        sm.signmuon_f8_matmul(*self.dq, *self.wt, cols, self.dy, self.space)
        sm.signmuon_f8_matmul(*self.dt, *self.yt, tokens, w.grad, self.space)
        sm.signmuon_rms_norm_backward(self.dy, self.dh, self.x, g1.weight.view(-1), self.rstd, self.dx, g1.grad, self.space,
                                      workers=workers)
        sm.signmuon_embedding_backward(self.ids, self.dx, 1.0, table.grad, self.space, accumulate=True)

    def clip(self):
        sm.signmuon_clip_grads(self.gradients, self.most, self.norms, self.space)

    def step(self):
        sm.signmuon_step(self.mats, self.params, self.step_space)

    def run(self):
        self.forward()
        self.backward()
        self.clip()
        self.step()


def check_norm(x, r, gamma, rstd, y, h):
    flat = lambda t: t.cpu().reshape(-1, t.shape[-1])  # noqa: E731
    stream = stored_sum(flat(x), None if r is None else flat(r))
    if h is not None:
        assert same_bits(flat(h), stream)
    want, tol, out, out_tol = normed(stream, gamma.cpu().view(-1), EPS)
    assert bool(((rstd.cpu().double().view(-1) - want).abs() <= 1.01 * tol).all())
    near(y.view(-1, y.shape[-1]), out, 1.01 * out_tol)
    return out, 1.01 * out_tol


def check_norm_grad(p, dy, dh, h, gamma, rstd, dx, dgamma):
    workers, _, _, cols = p.sizes
    flat = lambda t: t.cpu().reshape(-1, cols)  # noqa: E731
    want = backward_in_64(flat(dy), None if dh is None else flat(dh), flat(h), gamma.weight.cpu().view(-1),
                          rstd.cpu().view(-1), workers)
    near(dx.view(-1, cols), want[0], 1.01 * want[1])
    near(dgamma.view(workers, cols), want[2], 1.01 * want[3])


def check_pass(p):
    workers, tokens, vocab, cols = p.sizes
    table, w, g1, g2 = p.mats
    ids = p.ids.cpu()
    want = torch.where((ids >= 0)[..., None], table.weight.cpu().double()[ids.clamp(min=0)], 0.0)
    near(p.x, want, TINY)
    y, y_tol = check_norm(p.x, None, g1.weight, p.rstd, p.y, None)
    check_f8(p.yq[0].view(-1, p.yq[0].shape[-1]), p.yq[1].view(-1, p.yq[1].shape[-1]), y, y_tol, "e4m3")
    check_quant(p.yt, p.y.cpu().transpose(1, 2), E4)
    check_quant(p.wq, w.weight.cpu(), E4)
    check_quant(p.wt, w.weight.cpu().t(), E4)
    check_product(p.z, p.yq, p.wq, cols, E4, E4)
    check_norm(p.z, p.x, g2.weight, p.rstd2, p.y2, p.h)
    losses = losses_in_64(*logits_in_64(p.y2, table.weight, 1.0), p.targets, vocab)
    close(p.lse.flatten(), losses[0], losses[1], F32, "lse")
    close(p.loss.flatten(), losses[2], losses[3], F32, "loss")
    grads = gradients_in_64(p.y2, table.weight, p.targets, 1.0, p.lse, p.dloss, F32)
    close(p.dy2, grads[0], grads[1], p.act, "dy2")
    close(p.table_grad, grads[2], grads[3], F32, "the output layer's gradient")
    check_norm_grad(p, p.dy2, None, p.h, g2, p.rstd2, p.dh, g2.grad)
    check_quant(p.dq, p.dh.cpu(), E5)
    check_quant(p.dt, p.dh.cpu().transpose(1, 2), E5)
    check_product(p.dy, p.dq, p.wt, cols, E5, E4)
    check_product(w.grad, p.dt, p.yt, tokens, E5, E4)
    check_norm_grad(p, p.dy, p.dh, p.x, g1, p.rstd, p.dx, g1.grad)
    lookup, size, count = gradient_in_64(ids, p.dx.cpu(), 1.0, vocab)
    before = p.table_grad.cpu().double()
    # the lookup's sums, added once to what the output layer left
    near(table.grad, before + lookup, 1.002 * (count[..., None] + 1) * U * size + U * (before + lookup).abs())


SIZES = [(2, 300, 517, 200), (3, 5, 40, 64), (1, 70, 333, 129), (2, 33, 1000, 768)]


@pytest.mark.parametrize("workers,tokens,vocab,cols", SIZES)
@pytest.mark.parametrize("act", [F32, BF16])
@pytest.mark.parametrize("ns_iters", [0, 1])
def test_two_training_steps(workers, tokens, vocab, cols, act, ns_iters):
    p = Pass(workers, tokens, vocab, cols, act, ns_iters, most=0.5)
    p.reset()
    for i in range(2):
        p.feed(10 + i)
        before = [(m.momentum.cpu().numpy(), m.weight.cpu().numpy()) for m in p.mats]
        p.forward()
        p.backward()
        check_pass(p)
        given = [m.grad.cpu().view(workers, -1) for m in p.mats]
        p.clip()
        check_clip(given, p.most, p.norms, [m.grad.view(workers, -1) for m in p.mats])
        p.step()
        check_step(p, before, ns_iters)


@pytest.mark.parametrize("act", [F32, BF16])
def test_a_captured_step_replays_like_the_eager_one(act):
    p = Pass(2, 300, 517, 200, act, 1, most=0.5)

    def refresh(i):
        p.reset()
        p.feed(20 + i)

    outputs = [p.x, p.y, p.yq[0], p.z, p.h, p.y2, p.loss, p.dy2, p.dh, p.dy, p.dx, p.norms]
    for m in p.mats:
        outputs += [m.grad, m.momentum, m.packed, m.weight, m.vote_out]
    replays_like_eager(p.run, outputs, refresh)


def test_two_passes_on_two_streams():
    """Two models at once, each with its own buffers and workspaces."""
    passes = [Pass(2, 300, 517, 200, BF16, 1, most=0.5, seed=s) for s in (1, 2)]
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
