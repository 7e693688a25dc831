"""Host tests of the gated delta rule and the block norm (no GPU): exports, struct layouts, every refusal of the C
ABI's checks and of the Python entry points."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

import deterministic_fp32_gemm_amd as g
from deterministic_fp32_gemm_amd import _binding as B
from deterministic_fp32_gemm_amd import delta as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INCLUDE = os.path.join(ROOT, "include")


def declared():
    text = "".join(open(os.path.join(INCLUDE, h)).read() for h in ("sdm_gdr.h", "sdm_nrm.h"))
    return sorted(set(re.findall(r"SDM_GX_API\s+[\w\s]+?\*?\s?\b(sdm_\w+)\s*\(", text)))


def test_exports():
    assert declared() == sorted(D.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", D.DELTA_LIB_PATH], capture_output=True, text=True, check=True)
    exported = {ln.split()[-1] for ln in out.stdout.splitlines() if ln.split() and ln.split()[1] in ("T", "W")}
    assert exported == set(D.EXPORTS)


def test_struct_layouts(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text("""
#include <stdio.h>
#include <stddef.h>
#include "sdm_nrm.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu\\n", sizeof(sdm_rows_t), sizeof(sdm_gdr_args_t), offsetof(sdm_gdr_args_t, q),
         offsetof(sdm_gdr_args_t, d_o), offsetof(sdm_gdr_args_t, ds0), sizeof(sdm_gdr_step_args_t),
         offsetof(sdm_gdr_step_args_t, state), sizeof(sdm_nrm_args_t), offsetof(sdm_nrm_args_t, rstd));
  return 0;
}
""")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-Wall", "-Werror", "-pedantic", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    G, S, N = D.sdm_gdr_args_t, D.sdm_gdr_step_args_t, D.sdm_nrm_args_t
    assert got == [ctypes.sizeof(D.sdm_rows_t), ctypes.sizeof(G), G.q.offset, G.d_o.offset, G.ds0.offset, ctypes.sizeof(S),
                   S.state.offset, ctypes.sizeof(N), N.rstd.offset]


def rows(at, T, H, d):
    return D.sdm_rows_t(at, T * H * d, H * d, d)


def gdr(**kw):
    """A valid set of arguments at made-up addresses, with changes."""
    B_, T, Hk, Hv, dk, dv = 2, 70, 2, 4, 32, 48
    a = D.sdm_gdr_args_t(dtype=0, scale=1.0, B=B_, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, nseq=B_)
    at = 1 << 20
    for n, H, d in (("q", Hk, dk), ("k", Hk, dk), ("v", Hv, dv), ("g", Hv, 1), ("beta", Hv, 1), ("o", Hv, dv), ("d_o", Hv, dv),
                    ("d_q", Hk, dk), ("d_k", Hk, dk), ("d_v", Hv, dv), ("d_g", Hv, 1), ("d_beta", Hv, 1)):
        setattr(a, n, rows(at, T, H, d))
        at += 1 << 20
    for n in ("s0", "s_final", "ds_final", "ds0"):
        setattr(a, n, at)
        at += 1 << 20
    for n, v in kw.items():
        o, f = (a, n) if "." not in n else (getattr(a, n.split(".")[0]), n.split(".")[1])
        setattr(o, f, v)
    return a


def code(a, backward=0):
    return D.load().sdm_gdr_check(ctypes.byref(a), backward)


def test_gdr_accepts():
    for b in (0, 1):
        assert code(gdr(), b) == 0
        assert code(gdr(T=0), b) == 0
        assert code(gdr(s0=None, s_final=None, ds_final=None, ds0=None), b) == 0
    assert code(gdr(**{"q.data": 1 << 20, "k.data": 1 << 20})) == 0      # inputs may share memory
    assert code(gdr(B=1, nseq=5, cu_seqlens=64)) == 0


@pytest.mark.parametrize("change,status", [
    ({"dtype": 3}, B.SDM_GX_ERR_ARG), ({"dtype": -1}, B.SDM_GX_ERR_ARG), ({"B": 0}, B.SDM_GX_ERR_SHAPE),
    ({"T": -1}, B.SDM_GX_ERR_SHAPE), ({"T": 1 << 31}, B.SDM_GX_ERR_SHAPE), ({"T": 1 << 30}, B.SDM_GX_ERR_STRIDE),
    ({"Hk": 3}, B.SDM_GX_ERR_SHAPE), ({"Hk": 0}, B.SDM_GX_ERR_SHAPE), ({"Hv": 1}, B.SDM_GX_ERR_SHAPE),
    ({"dk": 0}, B.SDM_GX_ERR_SHAPE), ({"dk": 257}, B.SDM_GX_ERR_SHAPE), ({"dv": 257}, B.SDM_GX_ERR_SHAPE),
    ({"nseq": 3}, B.SDM_GX_ERR_SHAPE), ({"cu_seqlens": 64}, B.SDM_GX_ERR_SHAPE),
    ({"B": 1, "nseq": 0, "cu_seqlens": 64}, B.SDM_GX_ERR_SHAPE), ({"B": 1, "nseq": 1, "cu_seqlens": 66}, B.SDM_GX_ERR_ALIGN),
    ({"q.data": None}, B.SDM_GX_ERR_NULL), ({"beta.data": None}, B.SDM_GX_ERR_NULL), ({"o.data": None}, B.SDM_GX_ERR_NULL),
    ({"k.data": (1 << 20) + 2}, B.SDM_GX_ERR_ALIGN), ({"s0": (1 << 25) + 2}, B.SDM_GX_ERR_ALIGN),
    ({"v.token": -1}, B.SDM_GX_ERR_STRIDE), ({"v.head": 1 << 40}, B.SDM_GX_ERR_STRIDE),
    ({"o.head": 0}, B.SDM_GX_ERR_STRIDE), ({"o.token": 100}, B.SDM_GX_ERR_STRIDE), ({"o.batch": 1}, B.SDM_GX_ERR_STRIDE),
    ({"o.data": 3 << 20}, B.SDM_GX_ERR_OVERLAP), ({"s_final": 6 << 20}, B.SDM_GX_ERR_OVERLAP),
    ({"s_final": 13 << 20}, B.SDM_GX_ERR_OVERLAP),
])
def test_gdr_refuses(change, status):
    assert code(gdr(**change)) == status


@pytest.mark.parametrize("change,status", [
    ({"d_o.data": None}, B.SDM_GX_ERR_NULL), ({"d_g.data": None}, B.SDM_GX_ERR_NULL), ({"d_q.token": 1}, B.SDM_GX_ERR_STRIDE),
    ({"d_k.data": 8 << 20}, B.SDM_GX_ERR_OVERLAP), ({"d_v.data": 3 << 20}, B.SDM_GX_ERR_OVERLAP),
    ({"ds0": 15 << 20}, B.SDM_GX_ERR_OVERLAP), ({"d_beta.head": 0}, B.SDM_GX_ERR_STRIDE),
])
def test_gdr_backward_refuses(change, status):
    assert code(gdr(**change), 1) == status


def test_gdr_calls_refuse_before_any_device():
    lib = D.load()
    n = lib.sdm_gdr_workspace(ctypes.byref(gdr()), 0)
    assert n > 0 and lib.sdm_gdr_workspace(ctypes.byref(gdr()), 1) > n
    assert lib.sdm_gdr_workspace(ctypes.byref(gdr(dk=300)), 0) == B.SDM_GX_ERR_SHAPE
    assert lib.sdm_gdr_workspace(None, 0) == B.SDM_GX_ERR_ARG
    for fn in (lib.sdm_gdr_forward, lib.sdm_gdr_backward):
        assert fn(None, 1 << 30, n, None) == B.SDM_GX_ERR_ARG
        assert fn(ctypes.byref(gdr()), None, n, None) == B.SDM_GX_ERR_NULL
        assert fn(ctypes.byref(gdr()), (1 << 30) + 8, n, None) == B.SDM_GX_ERR_ALIGN
        assert fn(ctypes.byref(gdr()), 1 << 30, n - 1 if fn is lib.sdm_gdr_forward else n, None) == B.SDM_GX_ERR_LIMIT


def step(**kw):
    B_, T, Hk, Hv, dk, dv = 3, 1, 2, 4, 32, 48
    a = D.sdm_gdr_step_args_t(dtype=1, scale=1.0, B=B_, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, pool=5)
    at = 1 << 20
    for n, H, d in (("q", Hk, dk), ("k", Hk, dk), ("v", Hv, dv), ("g", Hv, 1), ("beta", Hv, 1), ("o", Hv, dv)):
        setattr(a, n, rows(at, T, H, d))
        at += 1 << 20
    a.state, a.slots = at, at + (1 << 24)
    for n, v in kw.items():
        o, f = (a, n) if "." not in n else (getattr(a, n.split(".")[0]), n.split(".")[1])
        setattr(o, f, v)
    return a


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"slots": None}, 0), ({"T": 0}, 0), ({"slots": None, "pool": 2}, B.SDM_GX_ERR_SHAPE),
    ({"pool": 0}, B.SDM_GX_ERR_SHAPE), ({"pool": 1 << 31}, B.SDM_GX_ERR_SHAPE), ({"dk": 257}, B.SDM_GX_ERR_SHAPE),
    ({"state": None}, B.SDM_GX_ERR_NULL), ({"state": (1 << 26) + 2}, B.SDM_GX_ERR_ALIGN), ({"slots": 2}, B.SDM_GX_ERR_ALIGN),
    ({"o.data": 0}, B.SDM_GX_ERR_NULL), ({"o.data": 1 << 20}, B.SDM_GX_ERR_OVERLAP), ({"state": 6 << 20}, B.SDM_GX_ERR_OVERLAP),
    ({"o.head": 1}, B.SDM_GX_ERR_STRIDE), ({"dtype": 7}, B.SDM_GX_ERR_ARG), ({"v.data": (1 << 28) + 1}, B.SDM_GX_ERR_ALIGN),
])
def test_step_checks(change, status):
    assert D.load().sdm_gdr_step_check(ctypes.byref(step(**change))) == status


def nrm(**kw):
    a = D.sdm_nrm_args_t(dtype=1, wtype=1, act=2, eps=1e-6, rows=10, D=100)
    at = 1 << 20
    for n in ("x", "o", "z", "w_post", "w_pre", "scale", "x_new", "y", "rstd", "dxn", "dy", "dx", "d_o", "dz", "dw_post",
              "dw_pre", "dscale"):
        setattr(a, n, at)
        at += 1 << 20
    for n in ("x", "o", "z", "xn", "y", "dxn", "dy", "dx", "do", "dz"):
        setattr(a, "ld_" + n, 100)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"rows": 0}, 0), ({"wtype": 0}, 0), ({"x": None}, 0), ({"w_pre": None, "y": None}, 0), ({"x_new": 1 << 20}, 0),
    ({"o": None, "z": None, "act": 0}, 0), ({"z": None, "act": 0}, 0),
    ({"dtype": 0, "wtype": 1}, B.SDM_GX_ERR_ARG), ({"wtype": 2}, B.SDM_GX_ERR_ARG), ({"act": 3}, B.SDM_GX_ERR_ARG),
    ({"eps": -1.0}, B.SDM_GX_ERR_ARG), ({"eps": float("nan")}, B.SDM_GX_ERR_ARG), ({"rows": -1}, B.SDM_GX_ERR_SHAPE),
    ({"D": 0}, B.SDM_GX_ERR_SHAPE), ({"D": 8193}, B.SDM_GX_ERR_SHAPE), ({"z": None}, B.SDM_GX_ERR_NULL),
    ({"act": 0}, B.SDM_GX_ERR_NULL), ({"o": None}, B.SDM_GX_ERR_NULL), ({"o": None, "w_pre": None}, B.SDM_GX_ERR_NULL),
    ({"o": None, "z": None, "act": 0, "x": None}, B.SDM_GX_ERR_NULL), ({"scale": None}, B.SDM_GX_ERR_NULL),
    ({"x_new": None}, B.SDM_GX_ERR_NULL), ({"y": None}, B.SDM_GX_ERR_NULL), ({"rstd": None}, B.SDM_GX_ERR_NULL),
    ({"ld_o": 99}, B.SDM_GX_ERR_STRIDE), ({"ld_y": 1 << 31}, B.SDM_GX_ERR_STRIDE), ({"x": (1 << 20) + 1}, B.SDM_GX_ERR_ALIGN),
    ({"w_pre": (1 << 28) + 1}, B.SDM_GX_ERR_ALIGN), ({"y": 2 << 20}, B.SDM_GX_ERR_OVERLAP), ({"y": 7 << 20}, B.SDM_GX_ERR_OVERLAP),
    ({"x_new": (1 << 20) + 200}, B.SDM_GX_ERR_OVERLAP), ({"x_new": 1 << 20, "ld_xn": 101}, B.SDM_GX_ERR_OVERLAP),
    ({"rstd": 1 << 20}, B.SDM_GX_ERR_OVERLAP), ({"x_new": 5 << 20}, B.SDM_GX_ERR_OVERLAP),
])
def test_nrm_checks(change, status):
    assert D.load().sdm_nrm_check(ctypes.byref(nrm(**change)), 0) == status


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"dxn": None}, 0), ({"dx": 10 << 20}, 0), ({"w_pre": None, "dy": None}, 0),
    ({"o": None, "z": None, "act": 0}, 0), ({"dy": None}, B.SDM_GX_ERR_NULL), ({"x_new": None}, B.SDM_GX_ERR_NULL),
    ({"dw_pre": None}, B.SDM_GX_ERR_NULL), ({"dz": None}, B.SDM_GX_ERR_NULL), ({"d_o": None}, B.SDM_GX_ERR_NULL),
    ({"dscale": None}, B.SDM_GX_ERR_NULL), ({"w_pre": None, "dxn": None}, B.SDM_GX_ERR_NULL),
    ({"o": None, "z": None, "act": 0, "dx": None}, B.SDM_GX_ERR_NULL), ({"dz": 13 << 20}, B.SDM_GX_ERR_OVERLAP),
    ({"dx": 11 << 20}, B.SDM_GX_ERR_OVERLAP), ({"dw_post": 4 << 20}, B.SDM_GX_ERR_OVERLAP), ({"ld_dz": 1}, B.SDM_GX_ERR_STRIDE),
])
def test_nrm_backward_checks(change, status):
    assert D.load().sdm_nrm_check(ctypes.byref(nrm(**change)), 1) == status


def test_nrm_workspace_refusals():
    lib = D.load()
    n = lib.sdm_nrm_workspace(ctypes.byref(nrm()))
    assert n > 0
    assert lib.sdm_nrm_workspace(ctypes.byref(nrm(D=0))) == B.SDM_GX_ERR_SHAPE
    assert lib.sdm_nrm_backward(ctypes.byref(nrm()), None, n, None) == B.SDM_GX_ERR_NULL
    assert lib.sdm_nrm_backward(ctypes.byref(nrm()), (1 << 30) + 4, n, None) == B.SDM_GX_ERR_ALIGN
    assert lib.sdm_nrm_backward(ctypes.byref(nrm()), 1 << 30, n - 1, None) == B.SDM_GX_ERR_LIMIT


def test_status_texts():
    for c in range(-11, 1):
        if c not in (B.SDM_GX_ERR_STEP, B.SDM_GX_ERR_PLAN):
            assert "unknown" not in D.load().sdm_delta_strerror(c).decode()


# ---- the Python entry points, on tensors that no GPU ever sees ------------------------------------------------------
def tensors(B_=1, T=4, Hk=1, Hv=2, dk=8, dv=8):
    r = torch.rand
    return dict(q=r(B_, T, Hk, dk), k=r(B_, T, Hk, dk), v=r(B_, T, Hv, dv), g=-r(B_, T, Hv), beta=r(B_, T, Hv))


@pytest.mark.parametrize("change,error", [
    ({}, ValueError),                                           # not on a GPU
    ({"q": None}, TypeError), ({"q": torch.rand(1, 4, 8)}, ValueError),
    ({"q": torch.rand(1, 4, 1, 8).double()}, TypeError), ({"v": torch.rand(1, 5, 2, 8)}, ValueError),
])
def test_python_refusals(change, error):
    t = {**tensors(), **change}
    with pytest.raises(error):
        g.gdr_forward(**t)
    with pytest.raises(error):
        g.gdr_backward(**t, do=torch.rand(1, 4, 2, 8))
    with pytest.raises(error):
        g.gdr_step(**t, state=torch.rand(1, 2, 8, 8))


@pytest.mark.parametrize("change", [
    {"act": "relu"}, {"z": None}, {"act": "none"}, {"o": None}, {"scale": None}, {"w_pre": torch.rand(7)},
    {"x": torch.rand(3, 9)}, {},
])
def test_python_norm_refusals(change):
    t = dict(x=torch.rand(3, 8), o=torch.rand(3, 8), z=torch.rand(3, 8), w_post=torch.rand(8), w_pre=torch.rand(8),
             scale=torch.rand(8), act="silu") | change
    with pytest.raises(ValueError):
        g.norm_forward(**t)
    act = t.pop("act")
    x = t.pop("x")
    with pytest.raises(ValueError):
        g.norm_backward(x, x, x, rstd=torch.rand(3, 2), act=act, **t)
