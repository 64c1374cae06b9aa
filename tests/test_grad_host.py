"""Host-side checks of the gradient operators: bad arguments are refused before
any launch (fake, never dereferenced device addresses), and the binding refuses
tensors of another type, shape, layout or device (no GPU needed)."""
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


def test_embedding_arguments(lib):
    names = "ids id_type table table_dtype tokens vocab cols scale y y_dtype stream".split()
    good = [A, 0, A, 0, 10, 20, 30, 1.0, A, 0, None]
    for change, status in [(dict(ids=None), EINVAL), (dict(table=None), EINVAL), (dict(y=None), EINVAL),
                           (dict(tokens=0), EINVAL), (dict(vocab=0), EINVAL), (dict(cols=-1), EINVAL),
                           (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
                           (dict(id_type=2), EDTYPE), (dict(table_dtype=2), EDTYPE), (dict(y_dtype=-1), EDTYPE),
                           (dict(ids=A + 8), EALIGN), (dict(table=A + 4), EALIGN), (dict(y=A + 2), EALIGN),
                           (dict(tokens=(1 << 25) + 1), ERANGE), (dict(vocab=(1 << 20) + 1), ERANGE),
                           (dict(cols=(1 << 20) + 1), ERANGE), (dict(vocab=1 << 20, cols=2048), ERANGE)]:
        assert calls_with(lib.signmuon_embedding, names, good, **change) == status, change


def test_embedding_backward_arguments(lib):
    names = ("ids id_type dy dy_dtype workers tokens vocab cols scale grad grad_dtype accumulate workspace "
             "workspace_bytes stream").split()
    good = [A, 1, A, 1, 2, 10, 20, 30, 1.0, A, 0, 0, *WS, None]
    need = sm.signmuon_embedding_workspace_bytes(2, 10, 20, 30)
    assert need >= 2 * 10 * 8
    for change, status in [(dict(ids=None), EINVAL), (dict(dy=None), EINVAL), (dict(grad=None), EINVAL),
                           (dict(workers=0), EINVAL), (dict(tokens=0), EINVAL), (dict(vocab=-5), EINVAL),
                           (dict(cols=0), EINVAL), (dict(scale=float("-inf")), EINVAL), (dict(accumulate=2), EINVAL),
                           (dict(id_type=-1), EDTYPE), (dict(dy_dtype=7), EDTYPE), (dict(grad_dtype=2), EDTYPE),
                           (dict(ids=A + 4), EALIGN), (dict(dy=A + 8), EALIGN), (dict(grad=A + 1), EALIGN),
                           (dict(workspace=WS[0] + 8), EALIGN), (dict(workspace=None), EWORKSPACE),
                           (dict(workspace_bytes=need - 1), EWORKSPACE), (dict(workers=256), ERANGE),
                           (dict(tokens=1 << 25), ERANGE), (dict(tokens=1 << 62), ERANGE),
                           (dict(vocab=1 << 20, cols=1 << 11), ERANGE)]:
        assert calls_with(lib.signmuon_embedding_backward, names, good, **change) == status, change


def test_embedding_workspace_sizes():
    size = sm.signmuon_embedding_workspace_bytes
    assert size(0, 1, 1, 1) == size(1, 0, 1, 1) == size(1, 1, 0, 1) == size(1, 1, 1, 0) == 0
    assert size(1, 4096, 100, 8) < size(1, 4097, 100, 8)  # several sorted runs: room to merge them
    # partial sums stay a small part of what a large batch reads
    assert size(8, 4096, 32000, 768) < 8 * 4096 * 768 * 2


def test_embedding_binding_refuses_other_tensors():
    ids, table = torch.zeros(2, 5, dtype=torch.int64), torch.zeros(7, 6)
    y = torch.zeros(2, 5, 6)
    with pytest.raises(TypeError, match="ids"):
        sm.signmuon_embedding(ids.float(), table, 1.0, y)
    with pytest.raises(TypeError, match="table"):
        sm.signmuon_embedding(ids, table.half(), 1.0, y)
    with pytest.raises(ValueError, match="table"):
        sm.signmuon_embedding(ids, table[0], 1.0, y)
    with pytest.raises(ValueError, match="y: shape"):
        sm.signmuon_embedding(ids, table, 1.0, y[:, :, :5])
    with pytest.raises(ValueError, match="contiguous"):
        sm.signmuon_embedding(ids, torch.zeros(6, 7).t(), 1.0, y)
    with pytest.raises(ValueError, match="GPU memory"):
        sm.signmuon_embedding(ids, table, 1.0, y)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    grad = torch.zeros(2, 7, 6)
    with pytest.raises(ValueError, match="dy"):
        sm.signmuon_embedding_backward(ids, y[:1], 1.0, grad, ws)
    with pytest.raises(ValueError, match="grad"):
        sm.signmuon_embedding_backward(ids, y, 1.0, grad[:1].contiguous(), ws)
    with pytest.raises(ValueError, match="ids"):
        sm.signmuon_embedding_backward(ids[0], y, 1.0, grad, ws)
    with pytest.raises(ValueError, match="GPU memory"):
        sm.signmuon_embedding_backward(ids, y, 1.0, grad, ws)


def test_layer_norm_arguments(lib):
    names = "x x_dtype rows cols gamma beta eps y mean rstd stream".split()
    good = [A, 1, 10, 20, A, None, 1e-5, A, None, None, None]
    for change, status in [(dict(x=None), EINVAL), (dict(gamma=None), EINVAL), (dict(y=None), EINVAL),
                           (dict(rows=0), EINVAL), (dict(cols=0), EINVAL), (dict(eps=0.0), EINVAL),
                           (dict(eps=-1e-5), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(x_dtype=2), EDTYPE),
                           (dict(x=A + 2), EALIGN), (dict(gamma=A + 4), EALIGN), (dict(beta=A + 8), EALIGN),
                           (dict(y=A + 4), EALIGN), (dict(mean=A + 4), EALIGN), (dict(rstd=A + 12), EALIGN),
                           (dict(rows=(1 << 25) + 1), ERANGE), (dict(cols=(1 << 20) + 1), ERANGE)]:
        assert calls_with(lib.signmuon_layer_norm, names, good, **change) == status, change


def test_layer_norm_backward_arguments(lib):
    names = ("dy x x_dtype workers rows cols gamma mean rstd dx dgamma dbeta grad_dtype workspace workspace_bytes "
             "stream").split()
    good = [A, A, 0, 2, 1000, 20, A, A, A, A, A, A, 1, *WS, None]
    need = sm.signmuon_layer_norm_workspace_bytes(2, 1000, 20)
    assert need > 0
    for change, status in [(dict(dy=None), EINVAL), (dict(x=None), EINVAL), (dict(gamma=None), EINVAL),
                           (dict(mean=None), EINVAL), (dict(rstd=None), EINVAL),
                           (dict(dx=None, dgamma=None, dbeta=None), EINVAL), (dict(workers=0), EINVAL),
                           (dict(rows=0), EINVAL), (dict(cols=-1), EINVAL), (dict(x_dtype=2), EDTYPE),
                           (dict(grad_dtype=3), EDTYPE), (dict(dx=A + 8), EALIGN), (dict(dgamma=A + 4), EALIGN),
                           (dict(dbeta=A + 2), EALIGN), (dict(dy=A + 2), EALIGN), (dict(workspace=None), EWORKSPACE),
                           (dict(workspace_bytes=need - 1), EWORKSPACE), (dict(workspace=WS[0] + 4), EALIGN),
                           (dict(workers=256), ERANGE), (dict(rows=1 << 25), ERANGE), (dict(rows=1 << 62), ERANGE),
                           (dict(cols=1 << 21), ERANGE)]:
        assert calls_with(lib.signmuon_layer_norm_backward, names, good, **change) == status, change


def test_layer_norm_binding_refuses_other_tensors():
    x, gamma, y = torch.zeros(4, 6), torch.zeros(6), torch.zeros(4, 6)
    s = torch.zeros(4)
    with pytest.raises(TypeError, match="gamma"):
        sm.signmuon_layer_norm(x, gamma.bfloat16(), None, 1e-5, y)
    with pytest.raises(ValueError, match="beta"):
        sm.signmuon_layer_norm(x, gamma, gamma[:5], 1e-5, y)
    with pytest.raises(TypeError, match="y"):
        sm.signmuon_layer_norm(x, gamma, None, 1e-5, y.bfloat16())
    with pytest.raises(ValueError, match="mean"):
        sm.signmuon_layer_norm(x, gamma, None, 1e-5, y, torch.zeros(5))
    with pytest.raises(ValueError, match="contiguous"):
        sm.signmuon_layer_norm(torch.zeros(6, 4).t(), gamma, None, 1e-5, y)
    with pytest.raises(ValueError, match="GPU memory"):
        sm.signmuon_layer_norm(x, gamma, None, 1e-5, y)
    back = sm.signmuon_layer_norm_backward
    with pytest.raises(ValueError, match="workers"):
        back(y, x, gamma, s, s, x, None, None, None, workers=3)
    with pytest.raises(ValueError, match="dgamma"):
        back(y, x, gamma, s, s, x, torch.zeros(1, 6), None, None, workers=2)
    with pytest.raises(TypeError, match="dbeta"):
        back(y, x, gamma, s, s, x, torch.zeros(2, 6), torch.zeros(2, 6).bfloat16(), None, workers=2)
    with pytest.raises(TypeError, match="dy"):
        back(y.bfloat16(), x, gamma, s, s, x, None, None, None)


def test_f8_sizes():
    assert [sm.signmuon_f8_pitch(k) for k in (0, 1, 127, 128, 129, 1000)] == [0, 128, 128, 128, 256, 1024]
    assert [sm.signmuon_f8_scale_pitch(k) for k in (0, 1, 512, 513, 1024, 1025)] == [0, 4, 4, 8, 8, 12]
    size = sm.signmuon_f8_matmul_workspace_bytes
    assert size(0, 1, 1, 1) == size(1, 0, 1, 1) == size(1, 1, 0, 1) == size(1, 1, 1, 0) == 0
    assert size(1, 8192, 2304, 768) == 0  # enough tiles: k stays whole
    assert size(1, 128, 128, 8192) > 0    # one tile and a long k: in parts


def test_f8_quant_arguments(lib):
    names = "x x_dtype batch rows cols format q q_scale qt qt_scale stream".split()
    good = [A, 0, 2, 10, 20, 0, A, A, A, A, None]
    for change, status in [(dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(q_scale=None), EINVAL),
                           (dict(qt=None), EINVAL), (dict(qt_scale=None), EINVAL),
                           (dict(q=None, q_scale=None, qt=None, qt_scale=None), EINVAL), (dict(batch=0), EINVAL),
                           (dict(rows=0), EINVAL), (dict(cols=-3), EINVAL), (dict(x_dtype=2), EDTYPE),
                           (dict(format=2), EDTYPE), (dict(x=A + 2), EALIGN), (dict(q=A + 8), EALIGN),
                           (dict(q_scale=A + 4), EALIGN), (dict(qt=A + 1), EALIGN), (dict(qt_scale=A + 4), EALIGN),
                           (dict(batch=256), ERANGE), (dict(rows=(1 << 25) + 1), ERANGE), (dict(cols=1 << 40), ERANGE),
                           (dict(rows=1 << 25, cols=1 << 14), ERANGE)]:
        assert calls_with(lib.signmuon_f8_quant, names, good, **change) == status, change


def test_f8_matmul_arguments(lib):
    names = ("a a_scale a_format b b_scale b_format batch m n k b_shared out out_dtype workspace workspace_bytes "
             "stream").split()
    good = [A, A, 0, A, A, 1, 1, 128, 128, 8192, 0, A, 0, *WS, None]
    need = sm.signmuon_f8_matmul_workspace_bytes(1, 128, 128, 8192)
    for change, status in [(dict(a=None), EINVAL), (dict(a_scale=None), EINVAL), (dict(b=None), EINVAL),
                           (dict(b_scale=None), EINVAL), (dict(out=None), EINVAL), (dict(batch=0), EINVAL),
                           (dict(m=0), EINVAL), (dict(n=0), EINVAL), (dict(k=0), EINVAL), (dict(b_shared=2), EINVAL),
                           (dict(a_format=2), EDTYPE), (dict(b_format=-1), EDTYPE), (dict(out_dtype=2), EDTYPE),
                           (dict(a=A + 8), EALIGN), (dict(a_scale=A + 4), EALIGN), (dict(b=A + 4), EALIGN),
                           (dict(b_scale=A + 1), EALIGN), (dict(out=A + 2), EALIGN), (dict(workspace=None), EWORKSPACE),
                           (dict(workspace_bytes=need - 1), EWORKSPACE), (dict(workspace=WS[0] + 4), EALIGN),
                           (dict(batch=256), ERANGE), (dict(m=(1 << 25) + 1), ERANGE), (dict(k=(1 << 22) + 1), ERANGE),
                           (dict(m=1 << 25, n=1 << 25), ERANGE)]:
        assert calls_with(lib.signmuon_f8_matmul, names, good, **change) == status, change


def test_workspace_of_a_batch_and_of_its_rows_as_one_product():
    """Few rows each need none; as one product they would be summed in parts."""
    size = sm.signmuon_f8_matmul_workspace_bytes
    assert size(8, 16, 300, 4096) == 0 < size(1, 8 * 16, 300, 4096)
    assert size(1, 8 * 16, 300, 4096) % (8 * 16 * 300 * 4) == 0


def test_f8_binding_refuses_other_tensors():
    x = torch.zeros(3, 10, 20)
    q, s = sm.f8_empty((3, 10, 20), torch.float8_e4m3fn, "cpu")
    qt, st = sm.f8_empty((3, 20, 10), torch.float8_e4m3fn, "cpu")
    with pytest.raises(ValueError, match="neither"):
        sm.signmuon_f8_quant(x, None, None)
    with pytest.raises(ValueError, match="go together"):
        sm.signmuon_f8_quant(x, q, None)
    with pytest.raises(TypeError, match="q:"):
        sm.signmuon_f8_quant(x, q.view(torch.uint8), s)
    with pytest.raises(ValueError, match="qt: shape"):
        sm.signmuon_f8_quant(x, q, s, q, s)
    with pytest.raises(TypeError, match="formats differ"):
        sm.signmuon_f8_quant(x, q, s, qt.view(torch.float8_e5m2), st)
    with pytest.raises(TypeError, match="x"):
        sm.signmuon_f8_quant(x.half(), q, s)
    with pytest.raises(ValueError, match="GPU memory"):
        sm.signmuon_f8_quant(x, q, s, qt, st)
    out = torch.zeros(3, 10, 10)
    with pytest.raises(ValueError, match="a: shape"):
        sm.signmuon_f8_matmul(q, s, q, s, 200, out, None)
    with pytest.raises(ValueError, match="b: shape"):
        sm.signmuon_f8_matmul(q, s, q[:2].contiguous(), s[:2].contiguous(), 20, out, None)
    with pytest.raises(TypeError, match="out"):
        sm.signmuon_f8_matmul(q, s, q, s, 20, out.half(), None)
    with pytest.raises(TypeError, match="a_scale"):
        sm.signmuon_f8_matmul(q, s.float(), q, s, 20, out, None)
    with pytest.raises(ValueError, match="GPU memory"):
        sm.signmuon_f8_matmul(q, s, q, s, 20, out, None)


def test_f8_row_sizes_of_lengths_that_no_operand_has():
    for k in (0, -1, (1 << 25) + 1, (1 << 63) - 1, -(1 << 63)):
        assert sm.signmuon_f8_pitch(k) == sm.signmuon_f8_scale_pitch(k) == 0
    assert sm.signmuon_f8_pitch(1 << 25) == 1 << 25 and sm.signmuon_f8_scale_pitch(1 << 25) == 1 << 18
