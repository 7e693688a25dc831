"""The 16-bit feed-forward gradient without the rounding of dg and du (precise): what the host launches for it, the way through
torch's graph, and its error, which is that of rounding the result."""

import ctypes

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from deterministic_fp32_gemm_amd import block as L
from tests.block_ref import TYPES, act64, half, tiny
from tests.gpu_util import say
from tests.test_block_host import no_library  # noqa: F401
from tests.test_ffn_tiles import made, struct


@pytest.mark.parametrize("ty,precise,parts", [("bf16", 0, 1), ("bf16", 1, 2), ("f16", 1, 2), ("f16", -5, 2), ("f32", 1, 1)])
def test_what_is_launched(ty, precise, parts):
    a = struct(ty, 601, 801, 503)
    small = 2 * (601 + 503) * 503
    before = L.load().sdm_ffn_workspace(ctypes.byref(a), 1)
    a.precise = precise
    assert made("sdm_ffn_backward", a, 1)["grad"][0] == parts
    assert (L.load().sdm_ffn_workspace(ctypes.byref(a), 1) - before > small) == (parts == 2)


@pytest.mark.parametrize("precise", [False, True])
def test_through_the_graph(no_library, monkeypatch, precise):  # noqa: F811
    seen, real = [], L.ffn_backward
    monkeypatch.setattr(L, "ffn_backward", lambda *a, **kw: (seen.append(kw["precise"]), real(*a, **kw))[1])
    x = torch.zeros(2, 3, 8, requires_grad=True)
    sdm.ffn_forward(x, torch.zeros(5, 8), torch.zeros(5, 8), precise=precise).sum().backward()
    assert seen == [precise] and x.grad.shape == x.shape


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,F", [(300, 200, 150), (70, 1000, 130), (260, 520, 700), (700, 100, 90)])
@pytest.mark.parametrize("ty,act", [("bf16", "none"), ("f16", "silu"), ("bf16", "gelu")])
def test_error(ty, act, M, K, F):
    """The bound of test_ffn_small_weights.py, element by element; the call that rounds dg and du misses it."""
    say("ffn precise", ty, act, M, K, F)
    t = TYPES[ty]
    gen = torch.Generator().manual_seed(M + K)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, wg, wu, dh = r(M, K).to(t), (r(F, K) * K ** -0.5).to(t), (r(F, K) * K ** -0.5).to(t), r(M, F).to(t)
    g, u = (x.float() @ wg.float().t()), (x.float() @ wu.float().t())
    c = [v.cuda() for v in (dh, x, wg, wu)], (g.cuda(), u.cuda())
    got, rough = sdm.ffn_backward(*c[0], c[1], act=act, precise=True), sdm.ffn_backward(*c[0], c[1], act=act)
    leaf = [v.clone().requires_grad_() for v in c[0][1:]]
    X, G, W, DH, g, u = (v.double() for v in (x, wg, wu, dh, g, u))
    f, df, _ = act64(g, act)
    dg, du = DH * u * df, DH * f
    gate = (8 + 16 * (1 + g.abs())) * 2.0 ** -24
    edg = half(t) ** 2 * dg.abs() + gate * (DH * u).abs() + tiny(t)
    edu = half(t) ** 2 * du.abs() + gate * DH.abs() + tiny(t)
    eps = lambda n: (2 * n / 16 + 40) * 2.0 ** -23  # noqa: E731
    for have, other, (s, d) in zip(got, rough, (
            (dg @ G + du @ W, edg @ G.abs() + edu @ W.abs() + eps(2 * F) * (dg.abs() @ G.abs() + du.abs() @ W.abs())),
            (dg.t() @ X, edg.t() @ X.abs() + eps(M) * (dg.abs().t() @ X.abs())),
            (du.t() @ X, edu.t() @ X.abs() + eps(M) * (du.abs().t() @ X.abs())))):
        bound = (s.to(t).double() - s).abs() + 2 * d
        off = (have.double().cpu() - s).abs()
        assert (off <= bound).all(), f"{int((off > bound).sum())} of {off.numel()}, by up to {float((off / bound).max()):.3g} times the bound"
        assert ((other.double().cpu() - s).abs() > bound).any()
    torch.autograd.backward(sdm.ffn_forward(*leaf, act=act, precise=True), c[0][0])
    kept = sdm.ffn_forward(*c[0][1:], act=act, keep=True)[1]
    for v, w in zip(leaf, sdm.ffn_backward(*c[0], kept, act=act, precise=True)):
        assert torch.equal(v.grad, w)
