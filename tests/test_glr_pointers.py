"""Host tests: every pointer that the recurrence's kernels use is refused where it is not the device's, also for calls without
tokens, which read and write the states."""

import ctypes

import pytest

from deterministic_fp32_gemm_amd import _binding as B
from tests.block_stub import HOST, call
from tests.test_block_host import glr, glr_step

WS = 1 << 40


@pytest.mark.parametrize("T", [0, 300])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("backward", [0, 1])
def test_states_of_the_host_are_refused(backward, packed, T):
    more = {"B": 1, "nseq": 5, "cu_seqlens": 14 << 20} if packed else {}
    name = ("sdm_glr_forward", "sdm_glr_backward")[backward]

    def run(**kw):
        return call(name, ctypes.byref(glr(T=T, **{**more, **kw})), WS, 1 << 30, None)

    assert run()[0] == B.SDM_GX_OK
    used = (["h0", "h_final"], ["dh_final", "dh0"])[backward] + (["cu_seqlens"] if packed else [])
    tokens = (["x.data", "g.data", "z.data", "y.data", "marks"], ["x.data", "g.data", "z.data", "dy.data", "dx.data", "dg.data", "dz.data", "marks", "h0"])[backward]
    for field in used + (tokens if T else []):
        assert run(**{field: HOST}) == (B.SDM_GX_ERR_DEVICE, []), field
    if not T:       # nothing of them is touched
        for field in tokens:
            assert run(**{field: HOST})[0] == B.SDM_GX_OK, field


def test_step():
    for field in ("x.data", "g.data", "z.data", "y.data", "state", "slots"):
        assert call("sdm_glr_step", ctypes.byref(glr_step(**{field: HOST})), None) == (B.SDM_GX_ERR_DEVICE, []), field
        assert call("sdm_glr_step", ctypes.byref(glr_step(T=0, **{field: HOST})), None) == (B.SDM_GX_OK, [])
