"""Helpers for the tests of the gradient operators: output buffers between
guard bytes, rounding units, captured replays, and the library's own choices of
kernels."""
import ctypes

import torch

import sign_muon_step_amd as sm

DEV = torch.device("cuda:0")
GUARD = 1024
# half a step of each storage type, relative to the value
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -120  # below this, results may be subnormal or flushed


class Guarded:
    """A tensor whose memory lies between guard bytes; filled with 0xA5."""

    def __init__(self, shape, dtype, device=DEV):
        size = torch.empty(0, dtype=dtype).element_size()
        n = 1
        for s in shape:
            n *= s
        self.nbytes = n * size
        self.raw = torch.full((2 * GUARD + (self.nbytes + 15) // 16 * 16,), 0xA5, dtype=torch.uint8, device=device)
        self.t = self.raw[GUARD:GUARD + self.nbytes].view(dtype).view(shape)

    def check(self, name="buffer"):
        assert bool((self.raw[:GUARD] == 0xA5).all()), f"{name}: written before its start"
        assert bool((self.raw[GUARD + self.nbytes:] == 0xA5).all()), f"{name}: written past its end"


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[t.element_size()])


def same_bits(a, b):
    return torch.equal(bits(a), bits(b))


def capture(call):
    """`call` recorded into a graph on a side stream (not run)."""
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.synchronize()
    return g


def replays_like_eager(call, outputs, refresh, rounds=3):
    """A captured `call` replayed `rounds` times gives the eager call's bits;
    refresh(i) puts new inputs into the same buffers, with eager work and
    waits between the replays."""
    refresh(0)
    g = capture(call)
    for i in range(rounds):
        refresh(i)
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outputs]
        refresh(i)
        for t in outputs:
            t.view(torch.uint8).fill_(0x5A) if t.dtype.itemsize == 1 else t.fill_(7)
        refresh(i)
        g.replay()
        torch.cuda.synchronize()
        for t, w in zip(outputs, want):
            assert same_bits(t, w), f"replay {i} differs from the eager call"


class _Plan(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("tile", "splits", "chunk", "waves")]


def f8_plan(batch, m, n, k):
    """The library's own plan of an 8-bit product (csrc/grad_internal.h, F8Plan): which kernel and tile, the parts of k
    and their blocks, and the waves that share a tile's k where m is small. No GPU needed."""
    fn = sm.library()._ZN2sm7f8_planEllll
    fn.restype, fn.argtypes = _Plan, [ctypes.c_int64] * 4
    return fn(batch, m, n, k)


def embed_segment(workers, tokens, cols):
    """Sorted tokens that a wave of the table's gradient takes (csrc/grad_internal.h). No GPU needed."""
    fn = sm.library()._ZN2sm13embed_segmentEill
    fn.restype, fn.argtypes = ctypes.c_int32, [ctypes.c_int32, ctypes.c_int64, ctypes.c_int64]
    return fn(workers, tokens, cols)


class _LossTiles(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("tm", "tn", "splits")]


class _LossPlan(ctypes.Structure):
    _fields_ = ([(name, ctypes.c_int64) for name in ("piece", "pitch")] +
                [(name, _LossTiles) for name in ("logits", "dx", "dw")] +
                [(name, ctypes.c_bool) for name in ("few", "g32", "parts")] +
                [(name, ctypes.c_size_t) for name in ("x", "w", "partial", "state", "target", "row0", "row1", "row2", "g",
                                                      "sum", "part", "total")])


def loss_plan(tokens, vocab, cols, x_dtype, w_dtype):
    """The library's own plan of an output layer's loss (csrc/grad_internal.h, LossPlan): tiles and parts of k. No GPU
    needed. The types as the C interface numbers them, here and below."""
    fn = sm.library()._ZN2sm9loss_planElllii
    fn.restype, fn.argtypes = _LossPlan, [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    return fn(tokens, vocab, cols, x_dtype, w_dtype)


def loss_grad_plan(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype):
    """The same of its gradients."""
    fn = sm.library()._ZN2sm14loss_grad_planElllliiib
    fn.restype, fn.argtypes = _LossPlan, [ctypes.c_int64] * 4 + [ctypes.c_int] * 3 + [ctypes.c_bool]
    return fn(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype, True)
