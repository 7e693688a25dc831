"""Sizes past what one launch can hold are refused by the entry points, before any device call (no GPU)."""

import ctypes

import pytest

from deterministic_fp32_gemm_amd import _binding as B
from deterministic_fp32_gemm_amd import delta as D

FAR = 1 << 44       # made-up addresses, further apart than any operand is long


def operands(a, names, T, Hk, Hv, dk, dv):
    at = FAR
    for n in names:
        H, d = {"q": (Hk, dk), "k": (Hk, dk), "d_q": (Hk, dk), "d_k": (Hk, dk), "g": (Hv, 1), "beta": (Hv, 1),
                "d_g": (Hv, 1), "d_beta": (Hv, 1)}.get(n, (Hv, dv))
        setattr(a, n, D.sdm_rows_t(at, T * H * d, H * d, d))
        at += FAR
    return at


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("B_,T,Hk,Hv,dk,dv,held", [
    (1 << 18, 1, 32, 32, 16, 16, False),        # 2^23 scan workgroups of 512 threads
    ((1 << 18) - 1, 1, 32, 32, 16, 16, True),
    (1 << 16, 1, 32, 32, 200, 64, False),       # wide heads go 16 columns a workgroup
    (1, 1 << 30, 1, 1, 16, 16, False),          # 2^24 chunks
    (1, (1 << 29) - 64, 1, 1, 16, 16, True),    # 2^23 - 1 of them, of 512 threads in the gradient
])
def test_sequences(backward, B_, T, Hk, Hv, dk, dv, held):
    a = D.sdm_gdr_args_t(dtype=1, scale=1.0, B=B_, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, nseq=B_)
    at = operands(a, ("q", "k", "v", "g", "beta", "o", "d_o", "d_q", "d_k", "d_v", "d_g", "d_beta"), T, Hk, Hv, dk, dv)
    lib = D.load()
    n = lib.sdm_gdr_workspace(ctypes.byref(a), backward)
    assert n > 0
    call = lib.sdm_gdr_backward if backward else lib.sdm_gdr_forward
    status = call(ctypes.byref(a), at, n, None)
    assert (status == B.SDM_GX_ERR_LIMIT) == (not held), status
    assert status != B.SDM_GX_OK


@pytest.mark.parametrize("B_,Hv,dk,dv,held", [(1 << 19, 32, 16, 16, False), ((1 << 19) - 1, 32, 16, 16, True),
                                              (1 << 17, 32, 256, 256, False), (1 << 17, 31, 256, 256, True)])
def test_steps(B_, Hv, dk, dv, held):
    a = D.sdm_gdr_step_args_t(dtype=1, scale=1.0, B=B_, T=1, Hk=1, Hv=Hv, dk=dk, dv=dv, pool=1)
    at = operands(a, ("q", "k", "v", "g", "beta", "o"), 1, 1, Hv, dk, dv)
    a.state, a.slots = at, at + FAR
    status = D.load().sdm_gdr_step(ctypes.byref(a), None)
    assert (status == B.SDM_GX_ERR_LIMIT) == (not held), status
    assert status != B.SDM_GX_OK


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("dtype,parts", [(0, 3), (1, 1), (2, 2)])
@pytest.mark.parametrize("B_,T,Hk,Hv,dk,dv", [(2, 4096, 8, 16, 128, 128), (1, 65, 3, 3, 40, 57), (3, 1, 1, 5, 200, 256)])
def test_workspace_is_what_the_header_says(B_, T, Hk, Hv, dk, dv, dtype, parts, backward):
    a = D.sdm_gdr_args_t(dtype=dtype, scale=1.0, B=B_, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, nseq=B_)
    dkp, dvp = 64 if dk <= 64 else 128 if dk <= 128 else 256, (dv + 7) // 8 * 8
    head = 75008 + 8 * dvp * (dk + 64) + (512 * dk if Hv > Hk else 0) if backward else 50432
    want = B_ * -(-T // 64) * (Hv * head + Hk * 384 * parts * dkp)
    assert 0 <= D.load().sdm_gdr_workspace(ctypes.byref(a), backward) - want < 14 * 256


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("rows,ld,status", [
    (1 << 39, 1 << 30, B.SDM_GX_ERR_STRIDE),        # 2^69 elements: past what an address holds
    (1 << 32, (1 << 31) - 1, B.SDM_GX_ERR_STRIDE), (1 << 20, 1 << 20, B.SDM_GX_OK)])
def test_rows_past_an_address(rows, ld, status, backward):
    a = D.sdm_nrm_args_t(dtype=1, wtype=1, act=2, eps=1e-6, rows=rows, D=100)
    at = FAR
    for n in ("x", "o", "z", "w_post", "w_pre", "scale", "x_new", "y", "rstd", "dxn", "dy", "dx", "d_o", "dz", "dw_post",
              "dw_pre", "dscale"):
        setattr(a, n, at)
        at += FAR
    for n in ("x", "o", "z", "xn", "y", "dxn", "dy", "dx", "do", "dz"):
        setattr(a, "ld_" + n, ld)
    assert D.load().sdm_nrm_check(ctypes.byref(a), backward) == status
