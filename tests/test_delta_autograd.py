"""The delta entry points in torch's graph. Gradients are those of gdr_backward and norm_backward, whose values other tests
hold against the definitions: here they have to arrive, bit for bit, at the right tensors."""

import contextlib
import types

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from deterministic_fp32_gemm_amd import delta as D


def gdr(device, seed=0, B=2, T=70, Hk=2, Hv=4, dk=32, dv=24, ty=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(B, T, Hk, dk), dim=-1).to(ty) for _ in range(2))
    t = dict(q=q, k=k, v=r(B, T, Hv, dv).to(ty), g=-r(B, T, Hv).abs(), beta=torch.sigmoid(r(B, T, Hv)))
    return {n: x.to(device) for n, x in t.items()}


def norm(device, seed=0, rows=6, D_=40):
    gen = torch.Generator().manual_seed(seed)
    t = {n: torch.randn(rows, D_, generator=gen) for n in ("x", "o", "z")}
    t |= {n: 1 + 0.3 * torch.randn(D_, generator=gen) for n in ("w_post", "w_pre", "scale")}
    return {n: x.to(device) for n, x in t.items()}


def leaves(t):
    return {n: x.clone().requires_grad_() for n, x in t.items()}


# ---- without a GPU: the library replaced by one that computes nothing ------------------------------------------------
@pytest.fixture
def no_library(monkeypatch):
    lib = types.SimpleNamespace(**{n: (lambda *a: 256) if n.endswith("_workspace") else (lambda *a: 0) for n in D.EXPORTS})
    monkeypatch.setattr(D, "load", lambda: lib)
    monkeypatch.setattr(D, "_tensor", lambda t, *rest: t)
    monkeypatch.setattr(D, "_OnDevice", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(D, "_stream", lambda device: 0)
    monkeypatch.setattr(D, "_plans", D._Plans())


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "initial_state"])
def test_one_leaf_of_the_rule_is_enough(no_library, name):
    t = {**gdr("cpu"), "initial_state": torch.zeros(2, 4, 32, 24)}
    t[name].requires_grad_()
    o, s = sdm.gdr_forward(**t)
    assert o.requires_grad and s.requires_grad
    (o.sum() + s.sum()).backward()
    assert t[name].grad is not None and t[name].grad.shape == t[name].shape
    with torch.no_grad():
        o, s = sdm.gdr_forward(**t)
    assert not o.requires_grad and not s.requires_grad
    with torch.inference_mode():
        assert not sdm.gdr_forward(**t)[0].requires_grad


@pytest.mark.parametrize("name", ["x", "o", "z", "w_post", "w_pre", "scale"])
def test_one_leaf_of_the_norm_is_enough(no_library, name):
    t = norm("cpu")
    t[name].requires_grad_()
    x_new, y, rstd = sdm.norm_forward(**t)
    assert x_new.requires_grad and y.requires_grad and not rstd.requires_grad
    (x_new.sum() + y.sum()).backward()
    assert t[name].grad is not None and t[name].grad.shape == t[name].shape
    with torch.no_grad():
        assert not sdm.norm_forward(**t)[1].requires_grad


def test_the_step_is_an_error_in_a_backward_pass(no_library):
    t = gdr("cpu", T=1)
    t["v"].requires_grad_()
    state = torch.zeros(2, 4, 32, 24)
    o = sdm.gdr_step(**t, state=state)
    with pytest.raises(RuntimeError, match="gdr_step has no gradient"):
        o.sum().backward()
    wide = torch.zeros(2, 2, 4, 24)
    for out in (torch.empty(2, 1, 4, 24), wide[:, 1:]):
        got = sdm.gdr_step(**t, state=state, out=out)
        assert got is out
        with pytest.raises(RuntimeError, match="gdr_step has no gradient"):
            got.sum().backward()
    assert not state.requires_grad
    with torch.no_grad():
        assert not sdm.gdr_step(**t, state=state).requires_grad


def test_a_state_that_was_saved_and_then_stepped_is_an_error(no_library):
    t = gdr("cpu", T=1)
    state = torch.zeros(2, 4, 32, 24)
    leaf = torch.ones(2, 4, 32, 24, requires_grad=True)
    loss = (leaf * state).sum()
    sdm.gdr_step(**t, state=state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        sdm.gdr_step(**t, state=torch.zeros(2, 4, 32, 24))


def test_a_scale_that_requires_a_gradient_is_refused(no_library):
    t = gdr("cpu", T=1)
    scale = torch.tensor(0.5, requires_grad=True)
    with pytest.raises(ValueError, match="scale"):
        sdm.gdr_forward(**t, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        sdm.gdr_step(**t, state=torch.zeros(2, 4, 32, 24), scale=scale)
    with torch.no_grad():
        sdm.gdr_forward(**t, scale=scale)
    sdm.gdr_forward(**t, scale=scale.detach())


# ---- on the GPU -----------------------------------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [False, True])
def test_rule(ty, packed):
    t = gdr("cuda", B=1 if packed else 2, ty=ty)
    cu = torch.tensor([0, 10, 10, 70], dtype=torch.int32).cuda() if packed else None
    n = 3 if packed else 2
    gen = torch.Generator().manual_seed(5)
    s0, ds = (0.3 * torch.randn(n, 4, 32, 24, generator=gen).cuda() for _ in range(2))
    do = torch.randn(t["v"].shape, generator=gen).to(ty).cuda()
    want_o, want_s = sdm.gdr_forward(**t, initial_state=s0, scale=0.2, cu_seqlens=cu)
    want = sdm.gdr_backward(**t, do=do, initial_state=s0, dfinal_state=ds, scale=0.2, cu_seqlens=cu)
    p = leaves({**t, "initial_state": s0})
    o, s = sdm.gdr_forward(**p, scale=0.2, cu_seqlens=cu)
    assert torch.equal(o, want_o) and torch.equal(s, want_s)
    got = torch.autograd.grad((o, s), list(p.values()), (do, ds))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # either output alone, and without states
    for outs, d in (((0,), (do, None)), ((1,), (torch.zeros_like(do), ds))):
        made = sdm.gdr_forward(**p, scale=0.2, cu_seqlens=cu)
        got = torch.autograd.grad([made[i] for i in outs], list(p.values()), [(do, ds)[i] for i in outs])
        want = sdm.gdr_backward(**t, do=d[0], initial_state=s0, dfinal_state=d[1], scale=0.2, cu_seqlens=cu)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    del p["initial_state"]
    o, s = sdm.gdr_forward(**p, final_state=False, cu_seqlens=cu)
    assert s is None
    got = torch.autograd.grad(o, list(p.values()), do)
    for a, b in zip(got, sdm.gdr_backward(**t, do=do, cu_seqlens=cu)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_rule_through_views_and_a_sum():
    """q, k, v cut out of one leaf, a gate shared by all tokens, and the broadcast gradient of a sum."""
    t = gdr("cuda", Hk=4)
    flat = torch.cat([t["q"].flatten(2), t["k"].flatten(2), t["v"].flatten(2)], -1).requires_grad_()
    beta = torch.full((1, 1, 4), 0.5, device="cuda", requires_grad=True)
    q, k, v = flat.split([4 * 32, 4 * 32, 4 * 24], -1)
    o, _ = sdm.gdr_forward(q.unflatten(-1, (4, 32)), k.unflatten(-1, (4, 32)), v.unflatten(-1, (4, 24)), t["g"],
                           beta.expand(2, 70, 4))
    o.sum().backward()
    full = {**t, "beta": torch.full((2, 70, 4), 0.5, device="cuda")}
    dq, dk, dv, _, dbeta, _ = sdm.gdr_backward(**full, do=torch.ones_like(t["v"]))
    assert torch.equal(flat.grad, torch.cat([dq.flatten(2), dk.flatten(2), dv.flatten(2)], -1))
    assert torch.equal(beta.grad, dbeta.sum((0, 1), keepdim=True))


@pytest.mark.gpu
def test_second_gradients_are_an_error():
    p = leaves(gdr("cuda"))
    o, _ = sdm.gdr_forward(**p)
    (dq,) = torch.autograd.grad(o.square().sum(), p["q"], create_graph=True)
    with pytest.raises(RuntimeError):
        dq.sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
def test_norm(act):
    t = norm("cuda")
    if act == "none":
        t["z"] = None
    gen = torch.Generator().manual_seed(7)
    dxn, dy = (torch.randn(6, 40, generator=gen).cuda() for _ in range(2))
    xn, y, rstd = sdm.norm_forward(**t, act=act, eps=1e-5)
    order = ("x", "o", "z", "w_post", "w_pre", "scale")

    def run(t, outs, grads):
        p = {n: None if x is None else x.clone().requires_grad_() for n, x in t.items()}
        made = sdm.norm_forward(**p, act=act, eps=1e-5)
        need = [n for n in order if p[n] is not None]
        got = torch.autograd.grad([made[i] for i in outs], [p[n] for n in need], grads, allow_unused=True)
        return made, dict(zip(need, got))

    def same(got, want):
        for n, w in zip(order, want):
            if n in got:
                assert (got[n] is None) == (w is None), n
                assert w is None or torch.equal(got[n], w), n

    w = [t[n] for n in ("o", "z", "w_post", "w_pre", "scale")]
    made, got = run(t, (0, 1), (dxn, dy))
    assert all(torch.equal(a, b) for a, b in zip(made, (xn, y, rstd)))
    same(got, sdm.norm_backward(dxn, dy, xn, *w, rstd, act=act))
    same(run(t, (1,), (dy,))[1], sdm.norm_backward(None, dy, xn, *w, rstd, act=act))
    # y not used: the second norm's weight has no gradient
    alone = sdm.norm_backward(dxn, None, None, t["o"], t["z"], t["w_post"], None, t["scale"], rstd, act=act)
    same(run(t, (0,), (dxn,))[1], alone)
    # no second norm, no residual
    part = {**t, "x": None, "w_pre": None}
    xn2, _, rstd2 = sdm.norm_forward(**part, act=act, eps=1e-5)
    want = sdm.norm_backward(dxn, None, None, t["o"], t["z"], t["w_post"], None, t["scale"], rstd2, act=act)
    made, got = run(part, (0,), (dxn,))
    assert made[1] is None and torch.equal(made[0], xn2)
    same(got, want)


@pytest.mark.gpu
def test_second_norm_alone():
    t = norm("cuda")
    p = {n: t[n].clone().requires_grad_() for n in ("x", "w_pre")}
    x, y, rstd = sdm.norm_forward(p["x"], None, None, None, p["w_pre"], None, act="none")
    assert x is p["x"]
    dy = torch.randn(6, 40, generator=torch.Generator().manual_seed(1)).cuda()
    got = torch.autograd.grad((x, y), list(p.values()), (dy, dy))
    want = sdm.norm_backward(dy, dy, t["x"], None, None, None, t["w_pre"], None, rstd, act="none")
    # the residual's own gradient is added by torch here, by the kernel there: one float32 rounding apart
    assert torch.allclose(got[0], want[0], rtol=2.0 ** -22, atol=2.0 ** -22) and torch.equal(got[1], want[4])


@pytest.mark.gpu
def test_on_a_named_stream():
    t = gdr("cuda")
    want_o, _ = sdm.gdr_forward(**t)
    do = torch.randn(t["v"].shape, generator=torch.Generator().manual_seed(2)).cuda()
    want = sdm.gdr_backward(**t, do=do)
    p = leaves(t)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    o, _ = sdm.gdr_forward(**p, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    got = torch.autograd.grad(o, list(p.values()), do)
    torch.cuda.synchronize()
    assert torch.equal(o, want_o)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_captured():
    """A block's forward and backward captured through torch's graph, replayed on new inputs with eager passes between."""
    names = ("q", "k", "v", "g", "beta")

    def both(t, n):
        o, s = sdm.gdr_forward(*(t[x] for x in names))
        x_new, y, _ = sdm.norm_forward(n["x"], o.flatten(2).flatten(0, 1)[:, :40], n["z"], n["w_post"], n["w_pre"], n["scale"])
        need = [*(t[x] for x in names), *n.values()]
        loss = (x_new * x_new).sum() + (y * n["x"].detach()).sum() + s.square().sum()
        return x_new, y, s, *torch.autograd.grad(loss, need, allow_unused=True)

    def inputs(seed):
        n = norm("cuda", seed, rows=140)
        n.pop("o")
        return leaves(gdr("cuda", seed)), leaves(n)

    sets = [inputs(i) for i in range(3)]
    buf = inputs(0)
    want = [both(*s) for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(*buf)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(*buf)
    for s, w in list(zip(sets, want)) * 2:
        with torch.no_grad():
            for to, src in zip(buf, s):
                for n in to:
                    to[n].copy_(src[n])
        graph.replay()
        both(*s)
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)
