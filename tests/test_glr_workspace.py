"""Host tests of what the recurrence's forward call asks for: no queue, and no workspace for one, where the lengths cannot matter
or the queue's words are too many to be cleared in one launch."""

import ctypes

import pytest

from deterministic_fp32_gemm_amd import _binding as B
from deterministic_fp32_gemm_amd import block as L
from tests.block_stub import call, library
from tests.test_block_host import glr

TILE = 128


def packed(T, D, nseq):
    a = glr(B=1, T=T, D=D, nseq=nseq, cu_seqlens=1 << 44, act=0)
    for i, n in enumerate(("x", "g", "y")):
        setattr(a, n, L.sdm_seq_t((i + 1) << 40, T * D, D))
    for i, n in enumerate(("h0", "marks", "h_final")):
        setattr(a, n, (i + 8) << 40)
    return a


def walks(longest, tickets):
    """The kernel's own choice, of the longest run's tiles and the queue's tickets."""
    return 27 * longest <= 100 + 46 * tickets // 256


@pytest.mark.parametrize("T,D,nseq", [(16384, 4096, 4096), (16384, 4096, 20), (9001, 1001, 23), (9001, 1001, 400), (512, 64, 3),
                                      (600, 64, 3), (600, 4096, 3), (100000, 64, 5000), (100000, 64, 100)])
def test_packed(T, D, nseq):
    a, lib = packed(T, D, nseq), library()
    tiles, cblocks = -(-T // TILE), -(-D // 64)
    rows = T // TILE + nseq
    queue = tiles > 4 and not walks(tiles, rows * cblocks)      # may the longest run there can be make it the queue's?
    n = lib.sdm_glr_workspace(ctypes.byref(a), 0)
    assert n == (8 * (64 + rows * cblocks * 128) if queue else 0)
    # at most what a run of all tokens is worth: 1.3 KB a token, however many runs there are
    assert n <= 1300 * T + 1024
    status, notes = call("sdm_glr_forward", ctypes.byref(a), 1 << 43, n, None)
    assert status == B.SDM_GX_OK and notes == [("glr_forward", rows if queue else 0, cblocks, 0, 0)]


@pytest.mark.parametrize("D", [512, 64 * 140])
def test_more_words_than_a_launch_clears_are_walked(D):
    T = 1 << 30 if D == 512 else 62 << 20
    a = glr(B=1, nseq=1, T=T, D=D, act=0)
    for i, n in enumerate(("x", "g", "y")):
        setattr(a, n, L.sdm_seq_t((i + 1) << 42, T * D, D))
    for i, n in enumerate(("h0", "marks", "h_final")):
        setattr(a, n, (2 * i + 9) << 42)
    assert library().sdm_glr_workspace(ctypes.byref(a), 0) == 0
    assert call("sdm_glr_forward", ctypes.byref(a), None, 0, None) == (B.SDM_GX_OK, [("glr_forward", 0, D // 64, 0, 0)])
