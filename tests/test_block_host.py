"""Host tests of libsdm_block (no GPU): exports, struct layouts, every refusal of the C ABI's checks and of the Python entry
points, workspaces, the machine code, and the entry points in torch's graph with a library that computes nothing."""

import ctypes
import os
import re
import subprocess
import types

import pytest
import torch

import deterministic_fp32_gemm_amd as g
from deterministic_fp32_gemm_amd import _binding as B
from deterministic_fp32_gemm_amd import _build, _code_check
from deterministic_fp32_gemm_amd import block as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INCLUDE = os.path.join(ROOT, "include")
HEADERS = ("sdm_glr.h", "sdm_qnt.h", "sdm_ffn.h")


def test_exports():
    text = "".join(open(os.path.join(INCLUDE, h)).read() for h in HEADERS)
    declared = set(re.findall(r"SDM_GX_API\s+[\w\s]+?\*?\s?\b(sdm_\w+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", _build.BLOCK_LIB_PATH], capture_output=True, text=True, check=True)
    exported = {ln.split()[-1] for ln in out.stdout.splitlines() if ln.split() and ln.split()[1] in ("T", "W")}
    assert declared == set(L.EXPORTS) == exported


def test_struct_layouts(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text("""
#include <stdio.h>
#include <stddef.h>
#include "sdm_glr.h"
#include "sdm_qnt.h"
#include "sdm_ffn.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu %zu %zu %d %d\\n", sizeof(sdm_seq_t), sizeof(sdm_glr_args_t),
         offsetof(sdm_glr_args_t, marks), offsetof(sdm_glr_args_t, dh0), sizeof(sdm_glr_step_args_t),
         offsetof(sdm_glr_step_args_t, slots), sizeof(sdm_qnt_args_t), offsetof(sdm_qnt_args_t, scale), sizeof(sdm_ffn_args_t),
         offsetof(sdm_ffn_args_t, gate), offsetof(sdm_ffn_args_t, ld_dwu), SDM_E4M3, SDM_ACT_GELU);
  return 0;
}
""")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-Wall", "-Werror", "-pedantic", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    G, S, Q, F = L.sdm_glr_args_t, L.sdm_glr_step_args_t, L.sdm_qnt_args_t, L.sdm_ffn_args_t
    z = ctypes.sizeof
    assert got == [z(L.sdm_seq_t), z(G), G.marks.offset, G.dh0.offset, z(S), S.slots.offset, z(Q), Q.scale.offset, z(F),
                   F.gate.offset, F.ld_dwu.offset, L.SDM_E4M3, L.ACTS["gelu"]]


def test_machine_code():
    assert _code_check.verify(_build.BLOCK_LIB_PATH, _build.llvm(), _code_check.BLOCK_WAITS) > 500


def changed(a, kw):
    for n, v in kw.items():
        o, f = (a, n) if "." not in n else (getattr(a, n.split(".")[0]), n.split(".")[1])
        setattr(o, f, v)
    return a


def glr(**kw):
    """A valid set of arguments at made-up addresses, a MiB apart, with changes."""
    a = L.sdm_glr_args_t(dtype=1, gtype=0, act=2, B=2, T=300, D=40, nseq=2)
    at = 1 << 20
    for n in ("x", "g", "z", "y", "dy", "dx", "dg", "dz"):
        setattr(a, n, L.sdm_seq_t(at, 300 * 40, 40))
        at += 1 << 20
    for n in ("h0", "marks", "h_final", "dh_final", "dh0"):
        setattr(a, n, at)
        at += 1 << 20
    return changed(a, kw)


SHAPE, ARG, NULL, STRIDE = B.SDM_GX_ERR_SHAPE, B.SDM_GX_ERR_ARG, B.SDM_GX_ERR_NULL, B.SDM_GX_ERR_STRIDE
ALIGN, OVERLAP, LIMIT = B.SDM_GX_ERR_ALIGN, B.SDM_GX_ERR_OVERLAP, B.SDM_GX_ERR_LIMIT


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"T": 0}, 0), ({"h0": None, "marks": None, "h_final": None}, 0), ({"act": 0, "z.data": None}, 0), ({"gtype": 1}, 0),
    ({"x.data": 2 << 20}, 0), ({"B": 1, "nseq": 5, "cu_seqlens": 64}, 0),
    ({"dtype": 3}, ARG), ({"dtype": -1}, ARG), ({"gtype": 2}, ARG), ({"act": 3}, ARG), ({"act": -1}, ARG), ({"B": 0}, SHAPE),
    ({"T": -1}, SHAPE), ({"T": (1 << 30) + 1}, SHAPE), ({"B": 4, "nseq": 4, "T": 1 << 29}, SHAPE), ({"D": 0}, SHAPE), ({"D": 65537}, SHAPE),
    ({"nseq": 3}, SHAPE), ({"nseq": 0, "B": 1, "cu_seqlens": 64}, SHAPE), ({"cu_seqlens": 64}, SHAPE),
    ({"B": 1, "nseq": 1, "cu_seqlens": 66}, ALIGN), ({"x.data": None}, NULL), ({"z.data": None}, NULL), ({"y.data": None}, NULL),
    ({"g.data": (1 << 25) + 2}, ALIGN), ({"x.data": (1 << 25) + 1}, ALIGN), ({"h0": (1 << 25) + 2}, ALIGN), ({"marks": (1 << 25) + 1}, ALIGN),
    ({"x.token": -1}, STRIDE), ({"x.token": 1 << 31}, STRIDE), ({"g.batch": 1 << 40}, STRIDE), ({"y.token": 39}, STRIDE),
    ({"y.batch": 0}, STRIDE), ({"y.batch": 11999}, STRIDE), ({"T": 1 << 29, "x.token": 1 << 30}, STRIDE),
    ({"y.data": 1 << 20}, OVERLAP), ({"y.data": (3 << 20) + 200}, OVERLAP), ({"marks": 2 << 20}, OVERLAP), ({"h_final": 9 << 20}, OVERLAP),
    ({"h_final": 10 << 20}, OVERLAP),
])
def test_glr_checks(change, status):
    assert L.load().sdm_glr_check(ctypes.byref(glr(**change)), 0) == status


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"dh_final": None, "dh0": None, "h0": None}, 0), ({"act": 0, "z.data": None, "dz.data": None}, 0),
    ({"marks": None}, NULL), ({"dy.data": None}, NULL), ({"dx.data": None}, NULL), ({"dg.data": None}, NULL), ({"dz.data": None}, NULL),
    ({"dx.token": 1}, STRIDE), ({"dg.data": (1 << 25) + 2}, ALIGN), ({"dx.data": 5 << 20}, OVERLAP), ({"dz.data": 6 << 20}, OVERLAP),
    ({"dh0": 12 << 20}, OVERLAP), ({"dx.data": 10 << 20}, OVERLAP),
])
def test_glr_backward_checks(change, status):
    assert L.load().sdm_glr_check(ctypes.byref(glr(**change)), 1) == status


def test_glr_sizes():
    lib, r = L.load(), ctypes.byref
    assert lib.sdm_glr_marks(r(glr())) == 2 * 3
    assert lib.sdm_glr_marks(r(glr(B=1, nseq=5, cu_seqlens=64))) == 300 // 128 + 5
    assert lib.sdm_glr_workspace(r(glr()), 0) == 0
    big = glr(T=1 << 20)
    n = lib.sdm_glr_workspace(r(big), 0)
    assert n > 0 and lib.sdm_glr_workspace(r(big), 1) > 0
    for f in (lib.sdm_glr_marks, lambda a: lib.sdm_glr_workspace(a, 0)):
        assert f(None) == ARG and f(r(glr(D=0))) == SHAPE and f(r(glr(nseq=0))) == SHAPE
    for n_, v in (("x", 1), ("g", 2), ("z", 3), ("y", 4)):
        setattr(big, n_, L.sdm_seq_t(v << 32, 40 << 20, 40))
    big.marks, big.h0, big.h_final = 5 << 32, 6 << 32, 7 << 32
    assert lib.sdm_glr_forward(r(big), None, n, None) == NULL
    assert lib.sdm_glr_forward(r(big), (1 << 40) + 8, n, None) == ALIGN
    assert lib.sdm_glr_forward(r(big), 1 << 40, n - 1, None) == LIMIT
    assert lib.sdm_glr_forward(None, 1 << 40, n, None) == ARG
    many = glr(B=(1 << 20) - 1, nseq=(1 << 20) - 1, T=1, D=40000, h0=None, marks=None, h_final=None, act=0)
    for n_, v in (("x", 1), ("g", 2), ("y", 3)):
        setattr(many, n_, L.sdm_seq_t(v << 40, 40000, 40000))
    assert lib.sdm_glr_forward(r(many), None, 0, None) == LIMIT      # launches of 2^32 threads or more


def glr_step(**kw):
    a = L.sdm_glr_step_args_t(dtype=1, gtype=0, act=2, B=3, T=2, D=40, pool=5, state=5 << 20, slots=6 << 20)
    for i, n in enumerate(("x", "g", "z", "y")):
        setattr(a, n, L.sdm_seq_t((i + 1) << 20, 80, 40))
    return changed(a, kw)


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"slots": None}, 0), ({"T": 0}, 0), ({"act": 0, "z.data": None}, 0), ({"slots": None, "pool": 2}, SHAPE), ({"pool": 2}, 0),
    ({"pool": 0}, SHAPE), ({"pool": 1 << 31}, SHAPE), ({"D": 65537}, SHAPE), ({"state": None}, NULL), ({"state": (5 << 20) + 2}, ALIGN),
    ({"slots": 2}, ALIGN), ({"y.data": 0}, NULL), ({"y.data": 1 << 20}, OVERLAP), ({"state": 4 << 20}, OVERLAP), ({"state": 1 << 20}, OVERLAP),
    ({"slots": 5 << 20}, OVERLAP), ({"slots": 4 << 20}, OVERLAP), ({"y.token": 1}, STRIDE), ({"dtype": 7}, ARG), ({"gtype": 2}, ARG),
])
def test_glr_step_checks(change, status):
    assert L.load().sdm_glr_step_check(ctypes.byref(glr_step(**change))) == status


def qnt(**kw):
    a = L.sdm_qnt_args_t(dtype=1, wtype=1, eps=1e-6, rows=10, D=100, ld_x=100, ld_r=100, ld_xn=100, ld_q=100)
    for i, n in enumerate(("x", "r", "w", "x_new", "q", "scale")):
        setattr(a, n, (i + 1) << 20)
    return changed(a, kw)


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"rows": 0}, 0), ({"wtype": 0}, 0), ({"w": None}, 0), ({"r": None, "x_new": None}, 0), ({"x_new": 1 << 20}, 0),
    ({"x_new": 2 << 20}, 0), ({"dtype": 0, "wtype": 1}, ARG), ({"wtype": 2}, ARG), ({"dtype": 3}, ARG), ({"eps": -1.0}, ARG),
    ({"eps": float("nan")}, ARG), ({"rows": -1}, SHAPE), ({"rows": 1 << 40}, SHAPE), ({"D": 0}, SHAPE), ({"D": 16385}, SHAPE),
    ({"x": None}, NULL), ({"q": None}, NULL), ({"scale": None}, NULL), ({"x_new": None}, NULL), ({"ld_x": 99}, STRIDE),
    ({"ld_q": 99}, STRIDE), ({"ld_r": 1 << 31}, STRIDE), ({"rows": 1 << 39, "ld_x": 1 << 30}, STRIDE), ({"x": (1 << 20) + 1}, ALIGN),
    ({"w": (1 << 25) + 1}, ALIGN), ({"scale": (1 << 25) + 2}, ALIGN), ({"q": 1 << 20}, OVERLAP), ({"q": 4 << 20}, OVERLAP),
    ({"scale": 5 << 20}, OVERLAP), ({"scale": 3 << 20}, OVERLAP), ({"x_new": (1 << 20) + 200}, OVERLAP), ({"x_new": 3 << 20}, OVERLAP),
    ({"x_new": 1 << 20, "ld_xn": 101}, OVERLAP),
])
def test_qnt_checks(change, status):
    assert L.load().sdm_qnt_check(ctypes.byref(qnt(**change))) == status


def ffn(**kw):
    a = L.sdm_ffn_args_t(dtype=1, otype=1, act=2, M=100, K=72, F=88)
    for i, (n, ld) in enumerate((("x", 72), ("wg", 72), ("wu", 72), ("h", 88), ("gate", 88), ("up", 88), ("dh", 88), ("dx", 72), ("dwg", 72), ("dwu", 72))):
        setattr(a, n, (i + 1) << 20)
        setattr(a, "ld_" + n, ld)
    return changed(a, kw)


SMALL = {"dtype": 3, "otype": 1, "sx": 20 << 20, "sg": 21 << 20, "su": 22 << 20}


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"M": 0}, 0), ({"gate": None, "up": None}, 0), (SMALL, 0), ({**SMALL, "otype": 2}, 0), ({"act": 3}, 0), ({"ld_x": 90}, 0),
    ({"dtype": 4}, ARG), ({"dtype": -1}, ARG), ({"otype": 0}, ARG), ({**SMALL, "otype": 0}, ARG), ({"act": 4}, ARG), ({"sx": 64}, ARG),
    ({**SMALL, "su": None}, NULL), ({"M": -1}, SHAPE), ({"M": (1 << 21) + 1}, SHAPE), ({"K": 0}, SHAPE), ({"F": 0}, SHAPE), ({"K": (1 << 20) + 1}, SHAPE),
    ({"x": None}, NULL), ({"wu": None}, NULL), ({"h": None}, NULL), ({"gate": None}, NULL), ({"up": None}, NULL), ({"ld_x": 71}, STRIDE),
    ({"ld_h": 87}, STRIDE), ({"ld_wg": 1 << 31}, STRIDE), ({"x": (1 << 25) + 1}, ALIGN), ({"gate": (1 << 25) + 2}, ALIGN),
    ({**SMALL, "sg": (21 << 20) + 2}, ALIGN), ({"h": 1 << 20}, OVERLAP), ({"h": 2 << 20}, OVERLAP), ({"gate": 4 << 20}, OVERLAP),
    ({**SMALL, "sx": 4 << 20}, OVERLAP),
])
def test_ffn_checks(change, status):
    assert L.load().sdm_ffn_check(ctypes.byref(ffn(**change)), 0) == status


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"h": None}, 0), (SMALL, ARG), ({"M": 0}, SHAPE), ({"dh": None}, NULL), ({"gate": None}, NULL), ({"up": None}, NULL),
    ({"dx": None}, NULL), ({"dwu": None}, NULL), ({"ld_dh": 80}, STRIDE), ({"dx": 7 << 20}, OVERLAP), ({"dwg": 10 << 20}, OVERLAP),
    ({"dwg": 1 << 20}, OVERLAP),
])
def test_ffn_backward_checks(change, status):
    assert L.load().sdm_ffn_check(ctypes.byref(ffn(**change)), 1) == status


def test_ffn_workspaces():
    lib, r = L.load(), ctypes.byref
    size = lambda **kw: lib.sdm_ffn_workspace(r(ffn(**kw)), 0)  # noqa: E731
    # rows where they lie; few rows
    assert size() == 0 and size(dtype=0, otype=0) == 0 and size(M=3, x=(1 << 25) + 2) == 0
    assert size(x=(1 << 25) + 2) > 0 and size(ld_wg=73) > 0 and size(K=71) > 0
    n = lib.sdm_ffn_workspace(r(ffn()), 1)
    assert n > 0 and lib.sdm_ffn_workspace(r(ffn(F=0)), 1) == SHAPE
    odd = ffn(K=71)
    need = lib.sdm_ffn_workspace(r(odd), 0)
    assert lib.sdm_ffn_forward(r(odd), None, need, None) == NULL
    assert lib.sdm_ffn_forward(r(odd), (1 << 30) + 128, need, None) == ALIGN
    assert lib.sdm_ffn_forward(r(odd), 1 << 30, need - 1, None) == LIMIT
    assert lib.sdm_ffn_backward(r(ffn()), 1 << 30, n - 1, None) == LIMIT
    assert lib.sdm_ffn_backward(None, 1 << 30, n, None) == ARG
    # launches of 2^32 threads or more
    big = ffn(M=1 << 21, F=1 << 20, K=8, gate=None, up=None, ld_x=8, ld_wg=8, ld_wu=8, ld_h=1 << 20, wg=1 << 40, wu=1 << 41, h=1 << 44)
    assert lib.sdm_ffn_forward(r(big), None, 0, None) == LIMIT
    for c in (B.SDM_GX_OK, NULL, SHAPE, ALIGN, OVERLAP, STRIDE, LIMIT, B.SDM_GX_ERR_HIP, B.SDM_GX_ERR_DEVICE, ARG):
        assert "unknown" not in lib.sdm_block_strerror(c).decode()


# ---- the Python entry points ---------------------------------------------------------------------------------------
X, W = torch.zeros(2, 3, 8), torch.zeros(5, 8)


@pytest.mark.parametrize("call,error", [
    (lambda: g.glr_forward(None, X), TypeError), (lambda: g.glr_forward(X[0], X[0]), ValueError), (lambda: g.glr_forward(X, X), ValueError),
    (lambda: g.glr_forward(X, X, X), ValueError), (lambda: g.glr_forward(X, X, act="silu"), ValueError),
    (lambda: g.glr_forward(X, X, X, act="gelu"), ValueError), (lambda: g.glr_forward(X.double(), X), TypeError),
    (lambda: g.glr_step(X, X, None, X), ValueError),
    (lambda: g.norm_quant(X, None, None), ValueError), (lambda: g.norm_quant(X, X, W[0]), ValueError), (lambda: g.quant_rows(W[0]), ValueError),
    (lambda: g.quant_rows(W), ValueError), (lambda: g.quant_rows(W.double()), TypeError), (lambda: g.quant_rows("x"), TypeError),
    (lambda: g.norm_quant(W, None, torch.zeros(8, dtype=torch.half)), ValueError),
    (lambda: g.ffn_forward(X, W, None), TypeError), (lambda: g.ffn_forward(X, W, W), ValueError), (lambda: g.ffn_forward(X, W, W, act="relu"), ValueError),
    (lambda: g.ffn_forward(X[0, 0], W, W), ValueError), (lambda: g.ffn_forward(X, X, W), ValueError), (lambda: g.ffn_forward(X.double(), W, W), TypeError),
    (lambda: g.ffn_backward(None, X, W, W, (X, X)), TypeError), (lambda: g.ffn_backward(X, X, W, W, X), TypeError),
    (lambda: g.ffn_backward(X, X, W, W, None), TypeError),
])
def test_python_refusals(call, error):
    with pytest.raises(error):
        call()


@pytest.fixture
def no_library(monkeypatch):
    """A library that computes nothing, and no GPU."""
    size = {n: (lambda *a: 6) if n.endswith("_marks") else (lambda *a: 256) for n in L.EXPORTS if n.endswith(("_workspace", "_marks"))}
    monkeypatch.setattr(L, "load", lambda: types.SimpleNamespace(**{n: size.get(n, lambda *a: 0) for n in L.EXPORTS}))

    def tensor(t, name, shape, dtype=None, device=None):
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(shape)} required, got {tuple(t.shape)}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name}: {dtype} required, got {t.dtype}")
        return t

    monkeypatch.setattr(L, "_tensor", tensor)
    monkeypatch.setattr(L, "_call", lambda fn, what, dev, *args: None)
    monkeypatch.setattr(L, "_plans", L._Plans())
    monkeypatch.setattr(L.delta, "_increment_version", lambda tensors: None)


def test_shapes_that_do_not_fit(no_library):
    f8 = torch.float8_e4m3fn
    q, w8, s = X.to(f8), W.to(f8), torch.ones(5)
    for call, error in [
            (lambda: g.glr_forward(X, X[:, :2]), ValueError), (lambda: g.glr_forward(X, X.half()), TypeError),
            (lambda: g.glr_step(X, X, None, None), ValueError), (lambda: g.glr_forward(X, X, initial_state=torch.zeros(3, 8)), ValueError),
            (lambda: g.glr_forward(X, X, cu_seqlens=torch.tensor([0, 3], dtype=torch.int32)), ValueError),
            (lambda: g.glr_forward(X[:1], X[:1], cu_seqlens=torch.tensor([0, 3])), TypeError),
            (lambda: g.glr_forward(X[:1], X[:1], cu_seqlens=torch.zeros(1, dtype=torch.int32)), ValueError),
            (lambda: g.glr_step(X, X, None, torch.zeros(1, 8)), ValueError), (lambda: g.glr_step(X, X, None, torch.zeros(8, 4).t()), ValueError),
            (lambda: g.glr_step(X, X, None, torch.zeros(4, 8), slots=torch.zeros(3, dtype=torch.int32)), ValueError),
            (lambda: g.glr_step(X, X, None, torch.zeros(4, 8), slots=torch.zeros(2)), TypeError),
            (lambda: g.norm_quant(X, X[:1], W[0]), ValueError), (lambda: g.norm_quant(X.half(), None, W[0].bfloat16()), TypeError),
            (lambda: g.ffn_forward(X, W, W[:4]), ValueError), (lambda: g.ffn_forward(X[..., :7], W, W), ValueError),
            (lambda: g.ffn_forward(X, W, W.half()), TypeError), (lambda: g.ffn_forward(X, W, W, dtype=torch.half), TypeError),
            (lambda: g.ffn_forward(X, W, W, x_scale=torch.ones(2, 3)), ValueError), (lambda: g.ffn_forward(q, w8, w8), ValueError),
            (lambda: g.ffn_forward(q, w8, w8, x_scale=torch.ones(2, 3), gate_scale=s, up_scale=s[:4]), ValueError),
            (lambda: g.ffn_forward(q, w8, w8, x_scale=torch.ones(2, 3), gate_scale=s, up_scale=s, dtype=torch.float32), TypeError),
            (lambda: g.ffn_backward(torch.zeros(2, 3, 5), X, W, W, (torch.zeros(2, 3, 5), torch.zeros(2, 3, 4))), ValueError),
            (lambda: g.ffn_backward(torch.zeros(2, 3, 5).half(), X.half(), W.half(), W.half(), (torch.zeros(2, 3, 5).half(),) * 2), TypeError)]:
        with pytest.raises(error):
            call()
    assert g.ffn_forward(q, w8, w8, x_scale=torch.ones(2, 3), gate_scale=s, up_scale=s).dtype == torch.bfloat16


@pytest.mark.parametrize("name", ["x", "g", "z", "h0"])
def test_one_leaf_of_the_recurrence_is_enough(no_library, name):
    t = {n: torch.zeros(2, 3, 8) for n in ("x", "g", "z")} | {"h0": torch.zeros(2, 8)}
    t[name].requires_grad_()
    y, h, marks = g.glr_forward(t["x"], t["g"], t["z"], act="silu", initial_state=t["h0"])
    assert y.requires_grad and h.requires_grad and not marks.requires_grad
    (y.sum() + h.sum()).backward()
    assert t[name].grad is not None and t[name].grad.shape == t[name].shape
    with torch.no_grad():
        assert not g.glr_forward(t["x"], t["g"], t["z"], act="silu", initial_state=t["h0"])[0].requires_grad
    h = g.glr_forward(t["x"], t["g"], t["z"], act="silu", initial_state=t["h0"])[1]
    h.sum().backward()      # the last state alone


@pytest.mark.parametrize("i", [0, 1, 2])
def test_one_leaf_of_the_product_is_enough(no_library, i):
    t = [X.clone(), W.clone(), W.clone()]
    t[i].requires_grad_()
    h, kept = g.ffn_forward(*t, keep=True)
    assert h.requires_grad and not any(k.requires_grad for k in kept)
    h.sum().backward()
    assert t[i].grad.shape == t[i].shape
    assert not g.ffn_forward(*(v.detach() for v in t)).requires_grad


def test_what_has_no_gradient_says_so(no_library):
    x, state = X.clone().requires_grad_(), torch.zeros(4, 8)
    y = g.glr_step(x, X, None, state)
    with pytest.raises(RuntimeError, match="glr_step has no gradient"):
        y.sum().backward()
    with pytest.raises(RuntimeError, match="quant_rows has no gradient"):
        g.quant_rows(x)[1].sum().backward()
    with torch.no_grad():
        assert not g.glr_step(x, X, None, state).requires_grad and not g.norm_quant(x, X, W[0])[1].requires_grad
    f8 = torch.float8_e4m3fn
    s = torch.ones(5, requires_grad=True)
    h = g.ffn_forward(X.to(f8), W.to(f8), W.to(f8), x_scale=torch.ones(2, 3), gate_scale=s, up_scale=s)
    with pytest.raises(RuntimeError, match="8-bit operands has no gradient"):
        h.sum().backward()
