"""8-bit products whose waves and workgroups go round their loops more than once:
several groups of blocks a wave in the kernel of few rows, several tiles a
workgroup in the kernel of tiles. Every entry is compared with the 64-bit product
of the values that the operands stand for; the plan that a size is meant for is
asserted beside it.

Blocks of one row have scales of their own here, so that a block taken with
another one's scale shows."""
import pytest
import torch

import sign_muon_step_amd as sm
from gpu_util import announce
from grad_util import DEV, HALF_STEP, TINY, f8_plan, same_bits
from test_gpu_f8 import E4, E5, Guarded, size_of_groups, up

COMPUTE_UNITS = 256
BOTH = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def _name_the_case(request):
    if request.node.get_closest_marker("gpu") is None:
        yield
        return
    announce(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# one row and up to 32: (batch, m, n, k), groups of four blocks of the busiest and of the idlest wave
FEW_ROWS = [((1, 1, 4096, 11008), 3, 2), ((1, 3, 70, 9000), 3, 2), ((1, 16, 100, 20000), 5, 5),
            ((2, 5, 33, 9000), 3, 2), ((1, 17, 4096, 11008), 3, 2), ((1, 32, 11008, 4096), 2, 2),
            ((1, 32, 70, 9300), 3, 2), ((1, 31, 19, 4100), 2, 1)]

# several tiles a workgroup: (batch, m, n, k), tile, blocks, parts of k
TILES = [((1, 8192, 2304, 768), 128, 6, 1), ((1, 8190, 2303, 700), 128, 6, 1), ((1, 8192, 2304, 128), 128, 1, 1),
         ((1, 8190, 2303, 640), 128, 5, 1), ((1, 6000, 3000, 100), 128, 1, 1), ((40, 1600, 33, 131), 128, 2, 1),
         ((1, 7000, 5000, 1000), 128, 8, 1), ((1, 6000, 4004, 1030), 128, 9, 1),
         ((40, 47, 33, 12501), 128, 98, 25), ((40, 47, 32, 12501), 128, 98, 25),
         ((1, 9000, 9000, 2000), 256, 16, 1), ((1, 9000, 8997, 2000), 256, 16, 1), ((3, 3000, 3000, 600), 256, 5, 1),
         ((8, 131, 13503, 135), 256, 2, 1), ((8, 136, 4266, 10546), 256, 83, 3), ((40, 130, 995, 10306), 256, 81, 3)]


@pytest.mark.parametrize("sizes,most,least", FEW_ROWS)
def test_plan_of_few_rows(sizes, most, least):
    p, groups = f8_plan(*sizes), up(up(sizes[3], 128) // 128, 4) // 4
    assert p.tile == 16 and p.splits == 1
    assert -(-groups // p.waves) == most >= 2 and groups // p.waves == least


@pytest.mark.parametrize("sizes,tile,blocks,parts", TILES)
def test_plan_of_tiles(sizes, tile, blocks, parts):
    batch, m, n, k = sizes
    p = f8_plan(*sizes)
    assert (p.tile, up(k, 128) // 128, p.splits) == (tile, blocks, parts)
    tiles = batch * -(-m // tile) * -(-n // tile) * parts
    assert tiles > COMPUTE_UNITS * (1 if tile == 256 else 2)


def operand(batch, rows, k, fmt, seed):
    """(bytes, scales) as the library quantises them (compared bit for bit elsewhere), their
    values and block scales in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    blocks = up(k, 128) // 128
    x = torch.randn(batch, rows, k, generator=g, device=DEV)
    e = torch.randint(-5, 6, (batch, rows, blocks), generator=g, device=DEV)
    x *= torch.exp2(e.float()).repeat_interleave(128, -1)[..., :k]
    q, s = sm.f8_empty((batch, rows, k), fmt, DEV)
    sm.signmuon_f8_quant(x, q, s)
    scale = torch.exp2(s[..., :blocks].double() - 127)
    assert scale.unique().numel() > 5 or rows * blocks < 20
    return q, s, (q.double().unflatten(-1, (blocks, 128)) * scale[..., None]).flatten(-2), scale


def check(sizes, fa, fb, out_dtype):
    """2^-23 of the sizes' sum for each of k additions in fp32; for a BF16 result also the cut of
    each 8 consecutive k, at most 8 * 2^-13 of their largest product, which is at most their sizes'
    sum; half a step."""
    batch, m, n, k = sizes
    a, b = operand(batch, m, k, fa, 1), operand(batch, n, k, fb, 2)
    out = Guarded((batch, m, n), out_dtype)
    ws = Guarded((sm.signmuon_f8_matmul_workspace_bytes(batch, m, n, k),), torch.uint8)
    args = (a[0], a[1], b[0], b[1], k, out.t, ws.t if ws.nbytes else None)
    sm.signmuon_f8_matmul(*args)
    torch.cuda.synchronize()
    out.check("out")
    ws.check("workspace")
    got = out.t.clone()
    ga, gb = size_of_groups(a[0], a[3], fa), size_of_groups(b[0], b[3], fb)
    for i in range(batch):
        want = a[2][i] @ b[2][i].t().contiguous()
        tol = 2.0 ** -23 * k * (a[2][i].abs() @ b[2][i].abs().t().contiguous())
        if out_dtype == torch.bfloat16:
            tol += 8 * 2.0 ** -13 * (ga[i] @ gb[i].t().contiguous())
        tol += HALF_STEP[out_dtype] * (want.abs() + tol) + TINY
        assert bool(((got[i].double() - want).abs() <= tol).all()), f"batch entry {i}"
        if out_dtype == torch.float32:  # roundings of random sign add as their root, over the result's entries
            assert float((got[i].double() - want).norm() / want.norm()) <= 2.0 ** -23 * (2 * k) ** 0.5
    sm.signmuon_f8_matmul(*args)
    torch.cuda.synchronize()
    assert same_bits(out.t, got)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [s for s, _, _ in FEW_ROWS])
@pytest.mark.parametrize("fa,fb", [(E4, E4), (E5, E4)])
@pytest.mark.parametrize("out_dtype", BOTH)
def test_waves_of_several_groups(sizes, fa, fb, out_dtype):
    check(sizes, fa, fb, out_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [s for s, _, _, _ in TILES])
@pytest.mark.parametrize("fa,fb", [(E4, E4), (E4, E5)])
@pytest.mark.parametrize("out_dtype", BOTH)
def test_workgroups_of_several_tiles(sizes, fa, fb, out_dtype):
    check(sizes, fa, fb, out_dtype)
