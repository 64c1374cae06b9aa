"""Host-side checks of the norm, loss and clipping operators: bad arguments are
refused before any launch (fake, never dereferenced device addresses), and the
binding refuses tensors of another type, shape, layout or device (no GPU
needed)."""
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
