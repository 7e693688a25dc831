"""The gated feed-forward product on the GPU against its definition in 64 bits: few rows and many, types, ends of rows inside
a step, tiles and wavefronts, strides and alignment, scales, gradients, graphs."""

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from tests.block_ref import TYPES, act64, ffn, within
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def inputs(ty, M, K, F, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    t = TYPES[ty]
    return [v.to(t).cuda() for v in (r(M, K), r(F, K) * K ** -0.5, r(F, K) * K ** -0.5, 0.5 * r(M, F))]


def check(x, wg, wu, dh, act):
    h, kept = sdm.ffn_forward(x, wg, wu, act=act, keep=True)
    assert torch.equal(h, sdm.ffn_forward(x, wg, wu, act=act))
    grads = sdm.ffn_backward(dh, x, wg, wu, kept, act=act)
    got = dict(zip(("h", "g", "u", "dx", "dwg", "dwu"), (h, *kept, *grads)))
    for name, (v, bound) in ffn(x, wg, wu, act, x.dtype, dh=dh).items():
        within(got[name], v, bound, name)
    return got


# rows: one, around 16, 32, 48 and 64 (the last of few), around the tiles of 128 and 256; lengths around 8 values, a step of 64
# and 128, and odd ones
SHAPES = [(1, 1, 1), (1, 2048, 70), (16, 64, 16), (17, 300, 33), (33, 520, 40), (64, 1030, 17), (65, 64, 64), (127, 72, 65),
          (128, 128, 128), (129, 200, 136), (70, 7, 5), (257, 1111, 333), (300, 136, 520), (520, 1000, 264)]


@pytest.mark.parametrize("M,K,F", SHAPES)
@pytest.mark.parametrize("ty,act", [("f32", "gelu"), ("bf16", "silu"), ("f16", "sigmoid")])
def test_against_the_definition(ty, act, M, K, F):
    say("ffn", ty, act, M, K, F)
    check(*inputs(ty, M, K, F), act)


@pytest.mark.parametrize("ty,M,K,F", [("bf16", 3, 200, 5000), ("f32", 40, 130, 4100), ("f16", 5001, 65, 72), ("bf16", 64, 1030, 8200),
                                      ("f32", 3001, 33, 30)])
def test_long_sums_of_the_gradient(ty, M, K, F):
    """Few tiles with long sums: cut into parts that are joined."""
    say("ffn long", ty, M, K, F)
    check(*inputs(ty, M, K, F), "silu")


@pytest.mark.parametrize("M,K,F", [(1, 2048, 70), (5, 64, 128), (2, 128, 1856), (26, 157, 130), (70, 58, 300)])
@pytest.mark.parametrize("ty", ["bf16", "f16"])
def test_gradients_of_few_values(ty, M, K, F):
    """dg and du come in two parts there, each of which is off by half a step: half a step squared is left of their rounding."""
    say("ffn few values", ty, M, K, F)
    x, wg, wu, dh = inputs(ty, M, K, F)
    grads = sdm.ffn_backward(dh, x, wg, wu, sdm.ffn_forward(x, wg, wu, act="gelu", keep=True)[1], act="gelu")
    want = ffn(x, wg, wu, "gelu", x.dtype, dh=dh, parts=2)
    for name, got in zip(("dx", "dwg", "dwu"), grads):
        within(got, *want[name], name)


@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu", "gelu"])
def test_activations(ty, act):
    x, wg, wu, dh = inputs(ty, 100, 64, 72)
    check((4 * x.float()).to(x.dtype), wg, wu, dh, act)


@pytest.mark.parametrize("ty,M,K,F,act", [("bf16", 4096, 264, 2056, "silu"), ("f16", 2100, 512, 4100, "gelu"), ("f32", 2049, 100, 4104, "silu")])
def test_large_tiles(ty, M, K, F, act):
    """Enough tiles of 256 x 256 for them to be taken."""
    say("ffn large", ty, M, K, F)
    check(*inputs(ty, M, K, F), act)


@pytest.mark.parametrize("M,K,F", SHAPES + [(4100, 400, 2064)])
def test_8_bits(M, K, F):
    say("ffn e4m3", M, K, F)
    x, wg, wu, _ = inputs("f32", M, K, F)
    (x, sx), (wg, sg), (wu, su) = (sdm.quant_rows(t) for t in (x, wg, wu))
    for act, dtype in (("silu", None), ("gelu", torch.float16)):
        h, kept = sdm.ffn_forward(x, wg, wu, act=act, x_scale=sx, gate_scale=sg, up_scale=su, dtype=dtype, keep=True)
        assert h.dtype == (dtype or torch.bfloat16)
        want = ffn(x, wg, wu, act, h.dtype, (sx, sg, su))
        for name, v in zip(("h", "g", "u"), (h, *kept)):
            within(v, *want[name], name)


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 200])
def test_strides_and_alignment(ty, M):
    """Rows inside wider ones, at any element; weights that lie one beside the other; an expanded gradient."""
    x, wg, wu, dh = inputs(ty, M, 72, 88)
    want = check(x, wg, wu, dh, "silu")
    for off in (1, 8):
        wide = torch.zeros(M, 96, dtype=x.dtype, device="cuda")
        wide[:, off:off + 72] = x
        both = torch.zeros(88, 168, dtype=x.dtype, device="cuda")
        both[:, off:off + 72], both[:, 80 + off:152 + off] = wg, wu
        X, G, W = wide[:, off:off + 72], both[:, off:off + 72], both[:, 80 + off:152 + off]
        h, kept = sdm.ffn_forward(X, G, W, keep=True)
        grads = sdm.ffn_backward(dh, X, G, W, kept)
        # the same operations on the same values in the same order
        for a, k in zip((h, *kept, *grads), ("h", "g", "u", "dx", "dwg", "dwu")):
            assert torch.equal(a, want[k]), k
    h = sdm.ffn_forward(x.t().contiguous().t(), wg, wu)
    assert torch.equal(h, want["h"])
    deep = sdm.ffn_forward(x.view(1, M, 1, 72), wg, wu)
    assert deep.shape == (1, M, 1, 88) and torch.equal(deep.view(M, 88), want["h"])
    one = dh[:1, :1].expand(M, 88)
    grads = sdm.ffn_backward(one, x, wg, wu, sdm.ffn_forward(x, wg, wu, keep=True)[1])
    again = sdm.ffn_backward(one.contiguous(), x, wg, wu, sdm.ffn_forward(x, wg, wu, keep=True)[1])
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("ty", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("M", [1, 40, 130])
def test_what_lies_behind_a_row_is_not_used(ty, M):
    """NaN beside the operands' rows and behind the last one, at lengths that end inside a piece, a step and a tile."""
    for K, F in ((72, 20), (136, 130), (37, 3)):
        x, wg, wu, _ = inputs("f32" if ty == "e4m3" else ty, M, K, F)
        s = {}
        if ty == "e4m3":
            (x, a), (wg, b), (wu, c) = (sdm.quant_rows(t) for t in (x, wg, wu))
            s = dict(x_scale=a, gate_scale=b, up_scale=c)
        want = sdm.ffn_forward(x, wg, wu, **s)
        views = []
        for t in (x, wg, wu):
            es = t.element_size()
            wide = torch.full((t.shape[0] + 300, (K * es + 15) // 16 * 16 // es + 16 // es), float("nan"), device="cuda").to(t.dtype)
            wide[:t.shape[0], :K] = t
            views.append(wide[:t.shape[0], :K])
        assert torch.isfinite(want).all() and torch.equal(sdm.ffn_forward(*views, **s), want)


def test_not_finite():
    """A row of x that is not finite spoils its row of h, a row of a weight its column."""
    for M in (5, 200):
        x, wg, wu, _ = inputs("bf16", M, 72, 88)
        want = sdm.ffn_forward(x, wg, wu)
        x[3, 70], wu[9, 0] = float("nan"), float("inf")
        h = sdm.ffn_forward(x, wg, wu)
        rows, cols = [i for i in range(M) if i != 3], [i for i in range(88) if i != 9]
        assert torch.isnan(h[3]).all() and not torch.isfinite(h[:, 9]).any()
        assert torch.equal(h[rows][:, cols], want[rows][:, cols])


def test_empty_batch():
    x, wg, wu, dh = inputs("bf16", 0, 72, 88)
    h, kept = sdm.ffn_forward(x, wg, wu, keep=True)
    assert h.shape == (0, 88)
    dx, dwg, dwu = sdm.ffn_backward(dh, x, wg, wu, kept)
    assert dx.shape == (0, 72) and dwg.shape == (88, 72) and not dwg.any() and not dwu.any()


@pytest.mark.parametrize("M", [9, 150])
def test_graph_and_stream(M):
    x, wg, wu, dh = inputs("f32", M, 100, 60)

    def step():
        h, kept = sdm.ffn_forward(x, wg, wu, keep=True)
        return (h, *sdm.ffn_backward(dh, x, wg, wu, kept))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, kept = sdm.ffn_forward(x, wg, wu, keep=True, stream=side)
    got = (h, *sdm.ffn_backward(dh, x, wg, wu, kept, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(1, 4):
        for t, new in zip((x, wg, wu, dh), inputs("f32", M, 100, 60, seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_gradients_through_the_graph_and_differences():
    x, wg, wu, dh = inputs("f32", 6, 10, 7)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
    h = sdm.ffn_forward(*leaves, act="gelu")
    h.backward(dh)
    _, kept = sdm.ffn_forward(x, wg, wu, act="gelu", keep=True)
    want = sdm.ffn_backward(dh, x, wg, wu, kept, act="gelu")
    assert all(torch.equal(t.grad, w) for t, w in zip(leaves, want))
    for i, name in enumerate(("x", "w_gate", "w_up")):
        gen = torch.Generator().manual_seed(i)
        d = torch.randn((x, wg, wu)[i].shape, generator=gen).double()

        def loss(s):
            t = [v.double().cpu() for v in (x, wg, wu)]
            t[i] = t[i] + s * d
            return (dh.double().cpu() * act64(t[0] @ t[1].t(), "gelu")[0] * (t[0] @ t[2].t())).sum()

        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        # the gradient is off by some 2^-20 of its terms, the difference by 1e-10 of third derivatives
        assert abs(slope - (want[i].double().cpu() * d).sum()) <= 1e-5 * (want[i].double().cpu().abs() * d.abs()).sum(), name
    with pytest.raises(RuntimeError):
        sdm.ffn_forward(*leaves, act="gelu", keep=True)[1][0].sum().backward()      # the kept products have no gradient


def test_a_block_as_it_is_used():
    """Recurrence, block norm, feed-forward: a training step through torch's graph, then the served form in 8 bits."""
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    B, T, D, F = 2, 150, 64, 96
    x, g = r(B, T, D), -r(B, T, D).abs()
    p = {"z": r(B, T, D), "wn": 1 + 0.1 * r(D), "wp": 1 + 0.1 * r(D), "s": 0.5 + 0.1 * r(D), "wg": r(F, D) / 8, "wu": r(F, D) / 8}

    def plain(x, g, z, wn, wp, s, wg, wu):
        h, out = torch.zeros_like(x[:, 0]), []
        for t in range(T):
            h = g[:, t].exp() * h + x[:, t]
            out.append(h)
        o = torch.stack(out, 1) * act64(z, "silu")[0]
        rms = lambda v, w: v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
        y = rms(x + s * rms(o, wn), wp)
        return act64(y @ wg.t(), "silu")[0] * (y @ wu.t())

    leaves = {"x": x, "g": g, **p}
    a = {k: v.clone().requires_grad_() for k, v in leaves.items()}
    o = sdm.glr_forward(a["x"], a["g"], a["z"], act="silu")[0]
    xn, y, _ = sdm.norm_forward(a["x"], o, None, a["wn"], a["wp"], a["s"], act="none")
    h = sdm.ffn_forward(y, a["wg"], a["wu"])
    dh = r(B, T, F)
    h.backward(dh)
    b = {k: v.double().cpu().requires_grad_() for k, v in leaves.items()}
    want = plain(**b)
    want.backward(dh.double().cpu())
    # some 400 roundings in a row at the most on any path, each 2^-24 of values near the norm of what they add up to
    assert (h.double().cpu() - want.detach()).norm() <= 400 * 2.0 ** -24 * want.detach().norm()
    for k in leaves:
        assert (a[k].grad.double().cpu() - b[k].grad).norm() <= 400 * 2.0 ** -24 * b[k].grad.norm(), k
    # served: the norm's output and the weights in 8 bits
    with torch.no_grad():
        q, sx, xq = sdm.norm_quant(x, p["s"] * o, p["wp"])
        (wg, sg), (wu, su) = sdm.quant_rows(p["wg"]), sdm.quant_rows(p["wu"])
        h8 = sdm.ffn_forward(q, wg, wu, x_scale=sx, gate_scale=sg, up_scale=su)
        ref = ffn(q.flatten(0, 1), wg, wu, "silu", h8.dtype, (sx.flatten(), sg, su))["h"]
        within(h8.flatten(0, 1), *ref, "served")


def test_captured():
    """The recurrence and the product captured forward and backward through torch's graph, replayed on new inputs with eager
    passes between."""
    T, D, F = 1500, 72, 104

    def made(seed):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        t = dict(x=r(1, T, D), g=-r(1, T, D).abs(), z=r(1, T, D), h0=r(1, D), wg=r(F, D) * D ** -0.5, wu=r(F, D) * D ** -0.5)
        dh, ds = r(1, T, F), r(1, D)
        return {k: v.cuda().requires_grad_() for k, v in t.items()}, dh.cuda(), ds.cuda()

    def both(t, dh, ds):
        y, s, _ = sdm.glr_forward(t["x"], t["g"], t["z"], act="silu", initial_state=t["h0"])
        h = sdm.ffn_forward(y, t["wg"], t["wu"], act="gelu")
        return (h, s, *torch.autograd.grad((h, s), list(t.values()), (dh, ds)))

    sets, buf = [made(i) for i in range(3)], made(0)
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
            for k, v in s[0].items():
                buf[0][k].copy_(v)
            buf[1].copy_(s[1])
            buf[2].copy_(s[2])
        graph.replay()
        both(*s)
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)
