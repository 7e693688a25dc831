"""Tensors with a tangent of torch's forward mode at every entry point of delta.py and block.py, with libraries that compute
nothing: such a tensor need not require a gradient, and a call that took it would lose its tangent without a word."""

import contextlib
import types

import pytest
import torch
import torch.autograd.forward_ad as fwd

import deterministic_fp32_gemm_amd as g
from deterministic_fp32_gemm_amd import block as L
from deterministic_fp32_gemm_amd import delta as D


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def lib(names):
        return types.SimpleNamespace(**{n: (lambda *a: 256) if n.endswith(("_workspace", "_marks")) else (lambda *a: 0) for n in names})

    for m in (D, L):
        monkeypatch.setattr(m, "load", lambda m=m: lib(m.EXPORTS))
        monkeypatch.setattr(m, "_tensor", lambda t, *rest: t)
        monkeypatch.setattr(m, "_plans", D._Plans())
    monkeypatch.setattr(D, "_OnDevice", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(D, "_stream", lambda device: 0)
    monkeypatch.setattr(D, "_increment_version", lambda tensors: None)
    monkeypatch.setattr(L, "_call", lambda fn, what, dev, *args: None)


def r(*shape):
    return torch.randn(*shape)


HEADS, X, W, S = (1, 3, 2, 8), (1, 3, 8), (5, 8), (1, 2, 8, 8)
CALLS = {
    "gdr_forward": (lambda q, k, v, a, b, s: g.gdr_forward(q, k, v, a, b, initial_state=s), [HEADS] * 3 + [(1, 3, 2)] * 2 + [S]),
    "gdr_backward": (lambda q, k, v, a, b, do, s, ds: g.gdr_backward(q, k, v, a, b, do, initial_state=s, dfinal_state=ds),
                     [HEADS] * 3 + [(1, 3, 2)] * 2 + [HEADS, S, S]),
    "gdr_step": (lambda q, k, v, a, b, s: g.gdr_step(q, k, v, a, b, s), [HEADS] * 3 + [(1, 3, 2)] * 2 + [S]),
    "norm_forward": (lambda x, o, z, a, b, s: g.norm_forward(x, o, z, a, b, s), [W] * 3 + [(8,)] * 3),
    "norm_backward": (lambda dx, dy, xn, o, z, a, b, s, rs: g.norm_backward(dx, dy, xn, o, z, a, b, s, rs), [W] * 5 + [(8,)] * 3 + [(5, 2)]),
    "glr_forward": (lambda x, a, z, h: g.glr_forward(x, a, z, act="silu", initial_state=h), [X] * 3 + [(1, 8)]),
    "glr_backward": (lambda x, a, z, dy, m, h, dh: g.glr_backward(x, a, z, dy, m, act="silu", initial_state=h, dfinal_state=dh),
                     [X] * 4 + [(256, 8), (1, 8), (1, 8)]),
    "glr_step": (lambda x, a, z, s: g.glr_step(x, a, z, s, act="silu"), [X] * 3 + [(1, 8)]),
    "norm_quant": (lambda x, y, w: g.norm_quant(x, y, w), [W, W, (8,)]),
    "quant_rows": (lambda x: g.quant_rows(x), [W]),
    "ffn_forward": (lambda x, a, b: g.ffn_forward(x, a, b), [X, W, W]),
    "ffn_backward": (lambda dh, x, a, b, m, n: g.ffn_backward(dh, x, a, b, (m, n)), [(1, 3, 5), X, W, W, (1, 3, 5), (1, 3, 5)]),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tangent_is_refused(name):
    call, shapes = CALLS[name]
    call(*(r(*s) for s in shapes))
    for i in range(len(shapes)):
        for grad in (False, True):
            with fwd.dual_level(), (contextlib.nullcontext() if grad else torch.no_grad()):
                t = [r(*s) for s in shapes]
                call(*t)                        # inside a level, but without a tangent
                t[i] = fwd.make_dual(t[i], r(*shapes[i]))
                assert not t[i].requires_grad
                with pytest.raises(RuntimeError, match=f"{name} has no forward-mode derivative"):
                    call(*t)
    call(*(r(*s) for s in shapes))


def test_scales_of_8_bit_operands():
    f8 = torch.float8_e4m3fn
    x, w = torch.zeros(X).to(f8), torch.zeros(W).to(f8)
    for i in range(3):
        with fwd.dual_level():
            s = [torch.ones(1, 3), torch.ones(5), torch.ones(5)]
            s[i] = fwd.make_dual(s[i], torch.ones_like(s[i]))
            with pytest.raises(RuntimeError, match="ffn_forward has no forward-mode derivative"):
                g.ffn_forward(x, w, w, x_scale=s[0], gate_scale=s[1], up_scale=s[2])


@pytest.mark.parametrize("name", ["norm_forward", "glr_forward", "ffn_forward"])
def test_through_torch_func(name):
    call, shapes = CALLS[name]
    t = [r(*s) for s in shapes]

    def first(v):
        out = call(v, *t[1:])
        return out if isinstance(out, torch.Tensor) else out[0]

    with pytest.raises(RuntimeError, match="no forward-mode derivative"):
        torch.func.jvp(first, (t[0],), (torch.ones_like(t[0]),))


def test_forward_over_reverse():
    """The gradient of a graph whose incoming gradient carries a tangent."""
    x = r(*X).requires_grad_()
    h = g.ffn_forward(x, r(*W), r(*W))
    with fwd.dual_level():
        dh = fwd.make_dual(torch.ones_like(h), torch.ones_like(h))
        with pytest.raises(RuntimeError):
            torch.autograd.grad(h, x, dh)
