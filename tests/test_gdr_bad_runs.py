"""Runs whose bounds no caller should pass: entries of cu_seqlens outside 0 .. T, or falling ones. The kernels clamp an
entry to the row and a run's end to its start.

Where every run is well defined after that, the results are those of the clamped bounds, within test_gdr.py's bounds. Where
runs overlap, values are unspecified, but nothing is written outside the outputs and the workspace, and no input changes:
here all operands lie in one allocation, between regions of a known pattern."""

import ctypes

import pytest
import torch

from deterministic_fp32_gemm_amd import delta as D
from tests import test_gdr as G

T = 130
MOST, LEAST = (1 << 31) - 1, -(1 << 31)
DEFINED = {"past the end": ([0, 7, 7, 1 << 30], [0, 7, 7, T]), "before the start": ([-5, 10, 20, 30], [0, 10, 20, 30]),
           "all past": ([MOST, MOST, MOST, MOST], [T, T, T, T]), "all before": ([LEAST, -1, LEAST, -7], [0, 0, 0, 0]),
           "whole range": ([LEAST, 64, 65, MOST], [0, 64, 65, T])}
UNDEFINED = [[0, 300, 100, 400], [130, 0, 130, 0], [100, 50, 130, 20], [MOST, LEAST, MOST, LEAST], [60, 130, 3, 130],
             [0, 130, 0, 130], [128, 64, 0, 129]]


@pytest.mark.gpu
@pytest.mark.parametrize("name", DEFINED)
@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
def test_defined_after_clamping(name, ty):
    bad, cu = DEFINED[name]
    print("defined", name, ty, flush=True)
    d = G.make(1, T, 1, 2, 64, 32, ty, nseq=3)
    cut = torch.tensor(bad, dtype=torch.int32).cuda()
    G.check_forward(d, ty, 1.0, cu, cu_seqlens=cut)
    if cu[0] < cu[-1]:
        G.check_backward(d, ty, 1.0, cu, cu_seqlens=cut)
    o, s = G.forward(d, 1.0, cu_seqlens=cut)
    held = torch.zeros(T, dtype=torch.bool)
    for a, b in zip(cu, cu[1:]):
        held[a:b] = True
    assert not o[0, ~held].any()
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b:
            assert torch.equal(s[i].cpu(), d["s0"][i])
    grads = G.backward(d, 1.0, cu_seqlens=cut)
    assert not any(x[0, ~held].any() for x in grads[:5])
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b:
            assert torch.equal(grads[5][i].cpu(), d["ds"][i])


class Arena:
    """One allocation of a known pattern, operands cut out of it with 64 KB of the pattern around each."""

    GUARD = 1 << 16

    def __init__(self, size, device="cuda"):
        self.bytes = (torch.arange(size, device=device) * 37 % 251).to(torch.uint8)
        self.pattern = self.bytes.clone()
        self.at, self.free = self.GUARD, []

    def take(self, nbytes):
        at = (self.at + 255) // 256 * 256
        self.at = at + nbytes + self.GUARD
        assert self.at <= self.bytes.numel()
        return at

    def put(self, t):
        """t's values, which must not change."""
        t = t.contiguous()
        n = t.numel() * t.element_size()
        at = self.take(n)
        for b in (self.bytes, self.pattern):
            b[at:at + n] = t.to(b.device).view(-1).view(torch.uint8)
        return self.bytes.data_ptr() + at

    def room(self, nbytes):
        """Space to be written."""
        at = self.take(nbytes)
        self.free.append((at, at + nbytes))
        return self.bytes.data_ptr() + at

    def damaged(self):
        other = self.bytes != self.pattern
        for a, b in self.free:
            other[a:b] = False
        return int(other.sum())


def test_a_stray_write_is_seen():
    """The regions around operands, and the operands that are read (on the CPU)."""
    arena = Arena(1 << 19, "cpu")
    base = arena.bytes.data_ptr()
    read, room = arena.put(torch.ones(10)) - base, arena.room(100) - base
    arena.bytes[room:room + 100] = 255
    assert arena.damaged() == 0
    for at in (room - 1, room + 100, read, read + 39, 0, room + 100 + Arena.GUARD - 1):
        kept = int(arena.bytes[at])
        arena.bytes[at] = kept ^ 1
        assert arena.damaged() == 1
        arena.bytes[at] = kept


@pytest.mark.gpu
@pytest.mark.parametrize("bad", UNDEFINED + [b for b, _ in DEFINED.values()], ids=str)
@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv,Hk,Hv", [(64, 32, 1, 2), (40, 72, 2, 2), (128, 128, 16, 32)])
def test_writes_stay_inside(bad, ty, dk, dv, Hk, Hv):
    print("bounds", bad, ty, dk, dv, Hk, Hv, flush=True)
    d = G.make(1, T, Hk, Hv, dk, dv, ty, nseq=3)
    es = d["q"].element_size()
    lib = D.load()
    for backward in (0, 1):
        a = D.sdm_gdr_args_t(dtype=D._dtype(d["q"], "q"), scale=1.0, B=1, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, nseq=3, cu_seqlens=4)
        n = lib.sdm_gdr_workspace(ctypes.byref(a), backward)
        arena = Arena(n + (64 << 20))
        rows = lambda at, H, c: D.sdm_rows_t(at, T * H * c, H * c, c)  # noqa: E731
        for name, H, c in (("q", Hk, dk), ("k", Hk, dk), ("v", Hv, dv), ("g", Hv, 1), ("beta", Hv, 1)):
            setattr(a, name, rows(arena.put(d[name]), H, c))
        a.cu_seqlens = arena.put(torch.tensor(bad, dtype=torch.int32))
        a.s0 = arena.put(d["s0"])
        if backward:
            a.d_o, a.ds_final = rows(arena.put(d["do"]), Hv, dv), arena.put(d["ds"])
            for name, H, c, e in (("d_q", Hk, dk, es), ("d_k", Hk, dk, es), ("d_v", Hv, dv, es), ("d_g", Hv, 1, 4),
                                  ("d_beta", Hv, 1, 4)):
                setattr(a, name, rows(arena.room(T * H * c * e), H, c))
            a.ds0 = arena.room(3 * Hv * dk * dv * 4)
        else:
            a.o, a.s_final = rows(arena.room(T * Hv * dv * es), Hv, dv), arena.room(3 * Hv * dk * dv * 4)
        ws = arena.room(n)
        torch.cuda.synchronize()
        call = lib.sdm_gdr_backward if backward else lib.sdm_gdr_forward
        assert call(ctypes.byref(a), ws, n, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert arena.damaged() == 0, ("backward" if backward else "forward", bad)
        assert (arena.bytes != arena.pattern).any()      # something was written, in its place
