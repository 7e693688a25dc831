"""Bounds of packed runs that are out of range and out of order, through the C entry points: every output, the marks, the states and
the workspace lie between guard regions inside larger allocations, and what lies around and between their rows keeps its bytes. Runs
that are walked, runs from the queue, and gradients in one part and in several."""

import ctypes

import pytest
import torch

from deterministic_fp32_gemm_amd import block
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

GUARD, FILL = 4096, 0xA5


class Guarded:
    """`rows` rows of `cols` float32 with a stride, between guards of one allocation, all filled with a byte."""

    def __init__(self, rows, cols, ld=None):
        self.rows, self.cols, self.ld = rows, cols, ld or cols
        self.bytes = torch.full((2 * GUARD + rows * self.ld * 4,), FILL, dtype=torch.uint8, device="cuda")
        self.ptr = self.bytes.data_ptr() + GUARD

    def whole(self):
        inside = self.bytes[GUARD:len(self.bytes) - GUARD].reshape(self.rows, self.ld * 4)
        return all(bool((b == FILL).all()) for b in (self.bytes[:GUARD], self.bytes[len(self.bytes) - GUARD:], inside[:, self.cols * 4:]))


# walked: few tiles; the queue's: one run could be long. Bounds below zero, past the end, falling, equal, and the type's extremes
LOW, HIGH = -2 ** 31, 2 ** 31 - 1
CASES = [(200, 12, [-5, 150, 90, 1000, 7]), (200, 70, [HIGH, LOW, HIGH, LOW, HIGH, 100]), (3000, 12, [-5, 1500, 90, 100000, 7]),
         (3000, 12, [0, 3000, 0, 3000, 0, 3000]), (3000, 130, [LOW, HIGH]), (3000, 12, [3000] * 9 + [0] * 70 + [2999, 2999, 5]),
         (9000, 5, [HIGH, 4000, LOW, 9001, 8999, 8999, 0, 9000]), (9000, 64, list(range(9000, 0, -90)) + [0] * 40)]


@pytest.mark.parametrize("T,D,cu", CASES)
def test_nothing_outside_is_written(T, D, cu):
    say("glr bad bounds", T, D, len(cu), cu[:4])
    lib, nseq, ld = block.load(), len(cu) - 1, D + 3
    gen = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    x, g, z, dy, h0, dh = r(T, D), -r(T, D).abs(), r(T, D), r(T, D), r(nseq, D), r(nseq, D)
    bounds = torch.tensor(cu, dtype=torch.int32, device="cuda")
    a = block.sdm_glr_args_t(dtype=0, gtype=0, act=2, B=1, T=T, D=D, nseq=nseq, cu_seqlens=bounds.data_ptr(), h0=h0.data_ptr(), dh_final=dh.data_ptr())
    for name, t in (("x", x), ("g", g), ("z", z), ("dy", dy)):
        setattr(a, name, block.sdm_seq_t(t.data_ptr(), T * D, D))
    out = {n: Guarded(T, D, ld) for n in ("y", "dx", "dg", "dz")}
    for name, o in out.items():
        setattr(a, name, block.sdm_seq_t(o.ptr, T * ld, ld))
    out |= {"marks": Guarded(lib.sdm_glr_marks(ctypes.byref(a)), D), "h_final": Guarded(nseq, D), "dh0": Guarded(nseq, D)}
    a.marks, a.h_final, a.dh0 = (out[n].ptr for n in ("marks", "h_final", "dh0"))
    stream = torch.cuda.current_stream().cuda_stream
    for backward, call in enumerate((lib.sdm_glr_forward, lib.sdm_glr_backward)):
        n = lib.sdm_glr_workspace(ctypes.byref(a), backward)
        ws = Guarded((n + 3) // 4, 1) if n else None
        assert call(ctypes.byref(a), ws.ptr if ws else None, n, stream) == 0
        torch.cuda.synchronize()
        for name, o in out.items():
            assert o.whole(), name
        assert ws is None or ws.whole()
    clamped = [min(max(c, 0), T) for c in cu]
    covered = torch.zeros(T, dtype=torch.bool)
    for lo, hi in zip(clamped, clamped[1:]):
        covered[lo:hi] = True
    for name in ("y", "dx", "dg", "dz"):        # tokens of no run keep their bytes
        rows = out[name].bytes[GUARD:-GUARD].reshape(T, ld * 4)
        assert (rows[~covered.cuda()] == FILL).all(), name
