"""Host-side checks of the norm, loss and clipping operators: bad arguments are
refused before any launch (fake, never dereferenced device addresses), and the
binding refuses tensors of another type, shape, layout or device (no GPU
needed)."""
import math
import random

import pytest
import torch

import sign_muon_step_amd as sm

A = 0x7f0000000000
WS = (0x7f1000000000, 1 << 40)
EINVAL, EDTYPE, EALIGN, EWORKSPACE, ERANGE = -1, -2, -3, -4, -6


@pytest.fixture(scope="module")
def lib():
    return sm.library()


def calls_with(fn, names, good, **change):
    args = dict(zip(names, good))
    for k in change:
        assert k in args
    args.update(change)
    return fn(*args.values())


def test_rms_norm_arguments(lib):
    names = "x residual x_dtype rows cols gamma eps h y format q q_scale rstd stream".split()
    good = [A, A, 1, 10, 20, A, 1e-5, A, A, 0, A, A, A, None]
    for change, status in [(dict(x=None), EINVAL), (dict(gamma=None), EINVAL), (dict(y=None, q=None, q_scale=None), EINVAL),
                           (dict(q=None), EINVAL), (dict(q_scale=None), EINVAL), (dict(residual=None), EINVAL),
                           (dict(rows=0), EINVAL), (dict(cols=0), EINVAL), (dict(eps=0.0), EINVAL),
                           (dict(eps=-1e-5), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(x_dtype=2), EDTYPE),
                           (dict(format=2), EDTYPE), (dict(format=-1), EDTYPE),
                           (dict(x=A + 2), EALIGN), (dict(residual=A + 8), EALIGN), (dict(gamma=A + 4), EALIGN),
                           (dict(h=A + 8), EALIGN), (dict(y=A + 4), EALIGN), (dict(q=A + 8), EALIGN),
                           (dict(q_scale=A + 1), EALIGN), (dict(rstd=A + 12), EALIGN),
                           (dict(rows=(1 << 25) + 1), ERANGE), (dict(cols=(1 << 20) + 1), ERANGE)]:
        assert calls_with(lib.signmuon_rms_norm, names, good, **change) == status, change


def test_rms_norm_backward_arguments(lib):
    names = "dy dh h x_dtype workers rows cols gamma rstd dx dgamma grad_dtype workspace workspace_bytes stream".split()
    good = [A, A, A, 0, 2, 1000, 20, A, A, A, A, 1, *WS, None]
    need = sm.signmuon_rms_norm_workspace_bytes(2, 1000, 20)
    assert need > 0
    for change, status in [(dict(dy=None), EINVAL), (dict(h=None), EINVAL), (dict(gamma=None), EINVAL),
                           (dict(rstd=None), EINVAL), (dict(dx=None, dgamma=None), EINVAL), (dict(workers=0), EINVAL),
                           (dict(rows=0), EINVAL), (dict(cols=-1), EINVAL), (dict(x_dtype=2), EDTYPE),
                           (dict(grad_dtype=3), EDTYPE), (dict(dx=A + 8), EALIGN), (dict(dgamma=A + 4), EALIGN),
                           (dict(dy=A + 2), EALIGN), (dict(dh=A + 2), EALIGN), (dict(h=A + 4), EALIGN),
                           (dict(rstd=A + 4), EALIGN), (dict(workspace=None), EWORKSPACE),
                           (dict(workspace_bytes=need - 1), EWORKSPACE), (dict(workspace=WS[0] + 4), EALIGN),
                           (dict(workers=256), ERANGE), (dict(rows=1 << 25), ERANGE), (dict(rows=1 << 62), ERANGE),
                           (dict(cols=1 << 21), ERANGE)]:
        assert calls_with(lib.signmuon_rms_norm_backward, names, good, **change) == status, change
    size = sm.signmuon_rms_norm_workspace_bytes
    assert size(0, 1, 1) == size(1, 0, 1) == size(1, 1, 0) == size(1, 1, 1) == 0


def test_rms_norm_binding_refuses_other_tensors():
    x, gamma, y, s = torch.zeros(4, 6), torch.zeros(6), torch.zeros(4, 6), torch.zeros(4)
    q, scale = sm.f8_empty((4, 6), torch.float8_e4m3fn, "cpu")
    norm = sm.signmuon_rms_norm
    with pytest.raises(TypeError, match="x: dtype"):
        norm(x.half(), None, gamma, 1e-5, y=y)
    with pytest.raises(TypeError, match="residual"):
        norm(x, x.bfloat16(), gamma, 1e-5, y=y)
    with pytest.raises(ValueError, match="residual"):
        norm(x, x[:3], gamma, 1e-5, y=y)
    with pytest.raises(TypeError, match="gamma"):
        norm(x, None, gamma.bfloat16(), 1e-5, y=y)
    with pytest.raises(TypeError, match="h: dtype"):
        norm(x, x, gamma, 1e-5, h=y.bfloat16(), y=y)
    with pytest.raises(ValueError, match="y: shape"):
        norm(x, None, gamma, 1e-5, y=y[:, :5])
    with pytest.raises(ValueError, match="rstd"):
        norm(x, None, gamma, 1e-5, y=y, rstd=s[:3])
    with pytest.raises(ValueError, match="go together"):
        norm(x, None, gamma, 1e-5, q=q)
    with pytest.raises(ValueError, match="q: shape"):
        norm(x, None, gamma, 1e-5, q=q[:, :64], q_scale=scale)
    with pytest.raises(ValueError, match="contiguous"):
        norm(torch.zeros(6, 4).t(), None, gamma, 1e-5, y=y)
    with pytest.raises(ValueError, match="GPU memory"):
        norm(x, None, gamma, 1e-5, y=y)
    back = sm.signmuon_rms_norm_backward
    with pytest.raises(ValueError, match="workers"):
        back(y, None, x, gamma, s, x, None, None, workers=3)
    with pytest.raises(ValueError, match="dgamma"):
        back(y, None, x, gamma, s, x, torch.zeros(1, 6), None, workers=2)
    with pytest.raises(TypeError, match="dy"):
        back(y.bfloat16(), None, x, gamma, s, x, None, None)
    with pytest.raises(TypeError, match="dh"):
        back(y, y.bfloat16(), x, gamma, s, x, None, None)
    with pytest.raises(TypeError, match="dgamma"):
        back(y, None, x, gamma, s, x, torch.zeros(1, 6).half(), None)
    with pytest.raises(ValueError, match="GPU memory"):
        back(y, None, x, gamma, s, y, None, None)


# ---------------------------------------------------------------------------
# Gradient norms and clipping
# ---------------------------------------------------------------------------
def entry(grad=A, out=A, n=10, dtype=0):
    return sm._Gradient(grad, out, n, dtype)


def test_clip_arguments(lib):
    names = "grads n_grads workers max_norm norms workspace workspace_bytes stream".split()

    def array(*entries):
        return (sm._Gradient * len(entries))(*entries)

    good = [array(entry(), entry(n=100000, dtype=1)), 2, 3, 1.0, A, *WS, None]
    need = lib.signmuon_grad_norm_workspace_bytes(good[0], 2, 3)
    assert need >= 3 * (1 + 7) * 8 + 3 * 4
    for change, status in [(dict(grads=None), EINVAL), (dict(n_grads=0), EINVAL), (dict(workers=0), EINVAL),
                           (dict(norms=None), EINVAL), (dict(max_norm=0.0), EINVAL), (dict(max_norm=-1.0), EINVAL),
                           (dict(max_norm=float("nan")), EINVAL), (dict(max_norm=float("inf")), EINVAL),
                           (dict(workers=256), ERANGE), (dict(n_grads=4097), ERANGE),
                           (dict(grads=array(entry(n=0), entry())), EINVAL),
                           (dict(grads=array(entry(), entry(n=1 << 31))), ERANGE),
                           (dict(grads=array(entry(grad=None), entry())), EINVAL),
                           (dict(grads=array(entry(out=None), entry())), EINVAL),
                           (dict(grads=array(entry(), entry(dtype=2))), EDTYPE),
                           (dict(grads=array(entry(), entry(grad=A + 4))), EALIGN),
                           (dict(grads=array(entry(), entry(out=A + 2))), EALIGN),
                           (dict(norms=A + 4), EALIGN), (dict(workspace=None), EWORKSPACE),
                           (dict(workspace_bytes=need - 1), EWORKSPACE), (dict(workspace=WS[0] + 8), EALIGN)]:
        assert calls_with(lib.signmuon_clip_grads, names, good, **change) == status, change
    names.remove("max_norm")
    del good[3]
    for change, status in [(dict(grads=None), EINVAL), (dict(norms=None), EINVAL), (dict(workers=-1), EINVAL),
                           (dict(workspace_bytes=need - 1), EWORKSPACE),
                           (dict(grads=array(entry(out=None), entry(dtype=-1))), EDTYPE),
                           (dict(grads=array(entry(out=None, grad=A + 8), entry())), EALIGN)]:
        assert calls_with(lib.signmuon_grad_norm, names, good, **change) == status, change


def test_gradients_refuses_other_tensors():
    a, b = torch.zeros(2, 6), torch.zeros(2, 3, 5)
    assert len(sm.Gradients([a, b])) == 2 and sm.Gradients([a, b]).workers == 2
    assert sm.signmuon_grad_norm_workspace_bytes(sm.Gradients([a, b])) > 0
    for grads, outs, error, match in [([], None, ValueError, "0 gradients"), ([a, b], [a], ValueError, "1 outs"),
                                      ([a, b[:1]], None, ValueError, r"grads\[1\]"),
                                      ([a.half()], None, TypeError, r"grads\[0\]"),
                                      ([torch.zeros(6, 2).t()], None, ValueError, "contiguous"),
                                      ([torch.zeros(2, 0)], None, ValueError, "entries"),
                                      ([torch.zeros(())], None, ValueError, "entries"),
                                      ([a], [a.bfloat16()], TypeError, r"outs\[0\]"),
                                      ([a], [torch.zeros(2, 5)], ValueError, r"outs\[0\]"),
                                      ([a, a], None, ValueError, "overlaps"),
                                      ([a, a], [torch.zeros(2, 6), a], ValueError, "overlaps"),
                                      ([a, b], [torch.zeros(2, 6), a.new_zeros(2, 3, 5).copy_(b)], None, "")]:
        if error is None:
            sm.Gradients(grads, outs)
        else:
            with pytest.raises(error, match=match):
                sm.Gradients(grads, outs)
    flat = torch.zeros(100)
    with pytest.raises(ValueError, match="overlaps"):
        sm.Gradients([a, torch.zeros(2, 20)], [flat[:12].view(2, 6), flat[8:48].view(2, 20)])
    sm.Gradients([a, a], [torch.zeros(2, 6), torch.zeros(2, 6)])  # read twice, written apart
    g, ws = sm.Gradients([a, b]), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="norms"):
        sm.signmuon_grad_norm(g, torch.zeros(3), ws)
    with pytest.raises(TypeError, match="norms"):
        sm.signmuon_clip_grads(g, 1.0, torch.zeros(2).double(), ws)
    with pytest.raises(ValueError, match="GPU memory"):
        sm.signmuon_clip_grads(g, 1.0, torch.zeros(2), ws)
    with pytest.raises(ValueError, match="GPU memory"):
        sm.signmuon_grad_norm(g, torch.zeros(2), ws)


# ---------------------------------------------------------------------------
# Softmax cross entropy of an output layer
# ---------------------------------------------------------------------------
SMALL = [(dict(tokens=0), EINVAL), (dict(vocab=0), EINVAL), (dict(cols=-1), EINVAL), (dict(scale=float("nan")), EINVAL),
         (dict(scale=float("inf")), EINVAL), (dict(x_dtype=2), EDTYPE), (dict(w_dtype=-1), EDTYPE),
         (dict(target_type=2), EDTYPE), (dict(x=A + 2), EALIGN), (dict(w=A + 8), EALIGN), (dict(targets=A + 4), EALIGN),
         (dict(workspace=None), EWORKSPACE), (dict(workspace=WS[0] + 8), EALIGN), (dict(tokens=(1 << 25) + 1), ERANGE),
         (dict(vocab=(1 << 20) + 1), ERANGE), (dict(cols=(1 << 20) + 1), ERANGE), (dict(vocab=1 << 20, cols=2048), ERANGE),
         (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(targets=None), EINVAL)]


def test_linear_cross_entropy_arguments(lib):
    names = ("x x_dtype w w_dtype targets target_type tokens vocab cols scale loss lse workspace workspace_bytes "
             "stream").split()
    good = [A, 1, A, 0, A, 1, 10, 1000, 20, 1.0, A, A, *WS, None]
    size = lib.signmuon_linear_cross_entropy_workspace_bytes
    need = size(10, 1000, 20, 1, 0)
    assert need > 0
    for change, status in SMALL + [(dict(loss=None, lse=None), EINVAL), (dict(loss=A + 4), EALIGN),
                                   (dict(lse=A + 8), EALIGN), (dict(workspace_bytes=need - 1), EWORKSPACE)]:
        assert calls_with(lib.signmuon_linear_cross_entropy, names, good, **change) == status, change
    assert size(0, 10, 10, 0, 0) == size(10, 0, 10, 0, 0) == size(10, 10, 0, 0, 0) == size(10, 10, 10, 2, 0) == 0
    # the logits of 8192 tokens would take 1.6 GB
    assert 0 < size(8192, 50257, 768, 1, 1) < 64 << 20


def test_linear_cross_entropy_backward_arguments(lib):
    names = ("x x_dtype w w_dtype targets target_type workers tokens vocab cols scale lse dloss dx dw grad_dtype "
             "accumulate workspace workspace_bytes stream").split()
    good = [A, 1, A, 1, A, 0, 2, 10, 1000, 20, 1.0, A, A, A, A, 0, 0, *WS, None]
    size = lib.signmuon_linear_cross_entropy_backward_workspace_bytes
    need = size(2, 10, 1000, 20, 1, 1, 0)
    assert need > 0
    for change, status in SMALL + [(dict(dx=None, dw=None), EINVAL), (dict(lse=None), EINVAL), (dict(dloss=None), EINVAL),
                                   (dict(accumulate=2), EINVAL), (dict(grad_dtype=2), EDTYPE), (dict(workers=0), EINVAL),
                                   (dict(workers=256), ERANGE), (dict(tokens=1 << 25), ERANGE), (dict(lse=A + 4), EALIGN),
                                   (dict(dloss=A + 8), EALIGN), (dict(dx=A + 2), EALIGN), (dict(dw=A + 2), EALIGN),
                                   (dict(workspace_bytes=need - 1), EWORKSPACE)]:
        assert calls_with(lib.signmuon_linear_cross_entropy_backward, names, good, **change) == status, change
    assert size(0, 10, 10, 10, 0, 0, 0) == size(1, 10, 10, 10, 0, 0, 3) == size(1, 10, 10, 10, 0, 5, 0) == 0


LOSS_SIZES = [(15892, 5428, 3544), (14467, 2202, 8104), (7910, 23213, 7534), (1, 1 << 20, 2047), (1 << 25, 1, 1),
              (1 << 23, 100, 64), (1 << 25, 65536, 64), (300, 3000, 1 << 19), (8192, 50257, 768), (65536, 32000, 4096)]


def _loss_sizes():
    rng = random.Random(5)
    some = [tuple(int(math.exp(rng.uniform(0, math.log(most)))) for most in (1 << 20, 1 << 17, 1 << 14)) for _ in range(20000)]
    return LOSS_SIZES + [(t, v, c) for t, v, c in some if v * c < 1 << 31]


def test_linear_cross_entropy_workspace_holds_no_logits(lib):
    """As the header bounds it: besides the operands' planes, what grows with tokens * vocab is held to a budget."""
    size = lib.signmuon_linear_cross_entropy_workspace_bytes
    for i, (t, v, c) in enumerate(_loss_sizes()):
        pitch, mb = (c + 7) // 8 * 8, 1 << 20
        for x, w in [(0, 0), (1, 1), (1, 0), (0, 1)][:4 if i < 2000 else 1]:
            planes = 0 if x and c % 8 == 0 else (2 if x else 6) * t * pitch
            weights = 0 if w and c % 8 == 0 else max(128 * mb, 256 * (2 if w else 6) * pitch)
            most = planes + weights + max(256 * mb, 32 * t) + 512 * mb + 12 * t + 8 * 256
            assert 0 < size(t, v, c, x, w) <= most, (t, v, c, x, w)


def test_linear_cross_entropy_backward_workspace_holds_no_logits(lib):
    """g is held to pieces of 1 GB, or to 256 columns of all tokens."""
    size = lib.signmuon_linear_cross_entropy_backward_workspace_bytes
    for i, (t, v, c) in enumerate(_loss_sizes()):
        pitch, gb = (c + 7) // 8 * 8, 1 << 30
        for x, w, grad in [(0, 0, 0), (1, 1, 0), (1, 1, 1), (1, 0, 0), (0, 1, 1)][:5 if i < 2000 else 1]:
            planes = (2 if x else 6) * t * pitch
            weights = 0 if w and c % 8 == 0 else max(gb, 256 * (2 if w else 6) * pitch)
            few = t <= 128
            g = max(gb, 256 * t * (2 if x and grad and not few else 4))
            sums = 4 * t * c if x else 0
            most = planes + weights + g + sums + max(gb, 4 * t * c) + 12 * t + 12 * 256
            for workers in {1, 8 if t % 8 == 0 else 1}:
                assert 0 < size(workers, t // workers, v, c, x, w, grad) <= most, (workers, t, v, c, x, w, grad)


def test_linear_cross_entropy_binding_refuses_other_tensors():
    x, w, ids = torch.zeros(2, 5, 6), torch.zeros(7, 6), torch.zeros(2, 5, dtype=torch.int64)
    s, ws = torch.zeros(2, 5), torch.zeros(1 << 20, dtype=torch.uint8)
    call = sm.signmuon_linear_cross_entropy
    for args, error, match in [((x.half(), w, ids, 1.0, s, s), TypeError, "x: dtype"),
                               ((x[:, :, :5], w, ids, 1.0, s, s), ValueError, "x: shape"),
                               ((x, w[0], ids, 1.0, s, s), ValueError, "w: 1 dim"),
                               ((x, w.double(), ids, 1.0, s, s), TypeError, "w: dtype"),
                               ((x, w, ids.float(), 1.0, s, s), TypeError, "targets"),
                               ((x, w, ids[:, :4], 1.0, s, s), ValueError, "x: shape"),
                               ((x, w, ids, 1.0, s[0], s), ValueError, "loss"),
                               ((x, w, ids, 1.0, s, s.bfloat16()), TypeError, "lse"),
                               ((x, torch.zeros(6, 7).t(), ids, 1.0, s, s), ValueError, "contiguous"),
                               ((x, w, ids, 1.0, s, s), ValueError, "GPU memory")]:
        with pytest.raises(error, match=match):
            call(*args, ws)
    back, dx, dw = sm.signmuon_linear_cross_entropy_backward, torch.zeros(2, 5, 6), torch.zeros(2, 7, 6)
    for args, error, match in [((x[0], w, ids[0], 1.0, s, s, dx, dw), ValueError, "targets"),
                               ((x, w, ids, 1.0, s[:1], s, dx, dw), ValueError, "lse"),
                               ((x, w, ids, 1.0, s, s.double(), dx, dw), TypeError, "dloss"),
                               ((x, w, ids, 1.0, s, s, dx.bfloat16(), dw), TypeError, "dx"),
                               ((x, w, ids, 1.0, s, s, dx, dw[:1]), ValueError, "dw"),
                               ((x, w, ids, 1.0, s, s, dx, dw.half()), TypeError, "dw"),
                               ((x, w, ids, 1.0, s, s, dx, dw), ValueError, "GPU memory")]:
        with pytest.raises(error, match=match):
            back(*args, ws)
