"""The gated linear recurrence where decays grow and fall: products of them over a tile, a group of tiles or a part leave float32
in both directions while the states stay far inside. Walked runs, tiles from the queue,
packed runs of either kind and gradients in parts, against the definition in 64 bits with the bounds of tests/block_ref.py
(8 roundings of 2^-24 a token, of what the recurrence over absolute values holds)."""

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from tests.block_ref import TYPES, glr, within
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def below(t, act, cu):
    """{name: what float32's smallest step costs}. A state under 2^-126 is rounded to a multiple of 2^-149, in each of at most 16
    roundings a token (its own, a map's and a power of two's), and what follows multiplies that by its decays: f_t <= a f_{t-1} +
    2^-145. So a state of the gradient of 1e-10 e^-96 = 2e-52 ("steep" from right to left) is zero, and e^96 times its error reaches
    the tokens before: 2^-145 e^96 = 0.01 there. dg multiplies exp(g) D, which has been rounded too, and the state before."""
    A = t["g"].double().exp()
    B, T, D = A.shape
    runs = [(b, 0, T) for b in range(B)] if cu is None else [(0, a, b) for a, b in zip(cu, cu[1:])]
    least = 2.0 ** -145
    met, d = torch.zeros(B, T, D, dtype=torch.float64), torch.zeros(B, T, D, dtype=torch.float64)
    last, first = (torch.full((len(runs), D), least, dtype=torch.float64) for _ in range(2))
    for i, (b, s, e) in enumerate(runs):
        for at in range(s, e):
            met[b, at] = last[i]
            last[i] = A[b, at] * last[i] + least
        for at in reversed(range(s, e)):
            d[b, at] = first[i] + least
            first[i] = A[b, at] * d[b, at] + least
    big = lambda v: v.double().abs()  # noqa: E731
    grad = glr(t["x"], t["g"], t["z"], act, t["h0"], cu, t["dy"], t["dh"])
    h = A * met + least
    states = glr(t["x"], t["g"], None, "none", t["h0"], cu)["y"][0]
    before = torch.zeros_like(states)
    before[:, 1:] = states[:, :-1]
    for i, (b, s, e) in enumerate(runs):
        if e > s:
            before[b, s] = t["h0"][i]
    gates = 1 if t["z"] is None else 1 + big(t["z"])        # bounds |act| and |act'|
    out = {"y": h * gates, "state": last, "dx": d, "dh0": first, "dg": (A * d + least) * (big(before) + met) + A * grad["dx"][0].abs() * met}
    return out if t["z"] is None else {**out, "dz": big(t["dy"]) * h * gates}


def check(t, act, cu=None):
    dev = {k: None if v is None else v.cuda() for k, v in t.items()}
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, h, marks = sdm.glr_forward(dev["x"], dev["g"], dev["z"], act=act, initial_state=dev["h0"], cu_seqlens=c)
    dx, dg, dz, dh0 = sdm.glr_backward(dev["x"], dev["g"], dev["z"], dev["dy"], marks, act=act, initial_state=dev["h0"],
                                       dfinal_state=dev["dh"], cu_seqlens=c)
    got = {"y": y, "state": h, "dx": dx, "dg": dg, "dz": dz, "dh0": dh0}
    floor = below(t, act, cu)
    for name, (v, bound) in glr(t["x"], t["g"], t["z"], act, t["h0"], cu, t["dy"], t["dh"]).items():
        assert torch.isfinite(v).all() and torch.isfinite(got[name]).all(), name
        within(got[name], v, bound + floor[name], name)


# three tiles are walked, 1300 tokens and more come from the queue; runs beside 600 of one token are walked, beside two taken
SIZES = [(1, 140, None), (2, 300, None), (1, 1300, None), (2, 2600, None), (1, None, [800] + [1] * 600), (1, None, [30, 2000, 500])]


def lengths(T, lens):
    cu = None if lens is None else [sum(lens[:i]) for i in range(len(lens) + 1)]
    return (T or cu[-1]), cu


@pytest.mark.parametrize("ty,act", [("f32", "none"), ("bf16", "silu")])
@pytest.mark.parametrize("B,T,lens", SIZES)
def test_a_level_that_wanders(B, T, lens, ty, act):
    """A state near e^S with S between -70 and 70 and steps of some 15: products up to e^140 and down to e^-140."""
    say("glr wandering", B, T, lens and len(lens), ty)
    T, cu = lengths(T, lens)
    n, D = B if lens is None else len(lens), 9
    gen = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    level = torch.zeros(B, T, D)
    at = torch.zeros(B, D)
    for i in range(T):
        at = (at + (15 * r(B, D)).clamp(-50, 50)).clamp(-70, 70)
        level[:, i] = at
    g = level - torch.cat([torch.zeros(B, 1, D), level[:, :-1]], 1)
    starts = torch.zeros(n, D) if lens is None else torch.stack([level[0, max(a - 1, 0)] if a else torch.zeros(D) for a in cu[:-1]])
    ends = level[:, -1] if lens is None else torch.stack([level[0, b - 1] for b in cu[1:]])
    t = dict(x=(level.exp() * r(B, T, D)).to(TYPES[ty]), g=g, z=None if act == "none" else r(B, T, D).to(TYPES[ty]),
             h0=starts.exp() * r(n, D), dy=((-level).exp() * r(B, T, D)).to(TYPES[ty]), dh=(-ends).exp() * r(n, D))
    check(t, act, cu)


@pytest.mark.parametrize("B,T,lens", SIZES)
@pytest.mark.parametrize("pattern", ["forget", "steep", "deep"])
def test_growth_that_ends(B, T, lens, pattern):
    """forget: a small state grows by e^100 and a gate of -inf ends it. steep: e^96 within 16 tokens and back. deep: down by e^120
    from a large state, and up again."""
    say("glr growth", B, T, lens and len(lens), pattern)
    T, cu = lengths(T, lens)
    n, D = B if lens is None else len(lens), 5
    g = torch.full((B, T, D), -0.01)
    for s in range(7, T - 120, 250):
        if pattern == "forget":
            g[:, s:s + 100], g[:, s + 100] = 1.0, -float("inf")
        elif pattern == "steep":
            g[:, s:s + 16], g[:, s + 20:s + 36] = 6.0, -6.0
        else:
            g[:, s:s + 10], g[:, s + 11:s + 21] = -12.0, 12.0
    gen = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    size = 1e25 if pattern == "deep" else 1e-10
    t = dict(x=torch.zeros(B, T, D), g=g, z=None, h0=size * r(n, D), dy=torch.zeros(B, T, D), dh=1e-10 * r(n, D))
    if pattern == "forget":
        t["x"][:, ::50] = 1e-10 * r(B, (T + 49) // 50, D)
        t["dy"][:, ::70] = 1e-10 * r(B, (T + 69) // 70, D)
    if pattern == "deep":
        t["dh"] *= 1e-15       # its product with the state is dg
    check(t, "none", cu)


def test_a_run_does_not_go_by_its_neighbours():
    """The same run alone in a packed row, beside many (walked), and beside a long one (from the queue)."""
    gen = torch.Generator().manual_seed(1)
    D, x, g = 6, torch.zeros(1, 300, 6), torch.full((1, 300, 6), 1.0)
    g[:, 100], g[:, 101:] = -float("inf"), 0.0
    x[:, 101:] = torch.randn(1, 199, 6, generator=gen)
    want = None
    for more in ([], [1] * 700, [4000]):
        lens = [300] + more
        X = torch.cat([x, torch.randn(1, sum(more), D, generator=gen)], 1).cuda()
        G = torch.cat([g, torch.full((1, sum(more), D), -0.1)], 1).cuda()
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
        y, h, _ = sdm.glr_forward(X, G, initial_state=torch.full((len(lens), D), 1e-10, device="cuda"), cu_seqlens=cu)
        assert torch.isfinite(y).all() and torch.isfinite(h).all()
        want = y[:, :300] if want is None else want
        assert ((y[:, :300] - want).abs() <= 300 * 8 * 2.0 ** -24 * (want.abs() + x.cuda().abs().cumsum(1))).all()


@pytest.mark.parametrize("T,lens", [(140, None), (1300, None), (None, [900, 400])])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 100.0])
def test_a_gate_that_is_not_finite_or_leaves_float32_stays_in_its_channel(value, T, lens):
    """It reaches the later states of its channel and run, the gradient of what comes before, and no others."""
    T, cu = lengths(T, lens)
    n, D, at = 1 if lens is None else len(lens), 6, 130
    gen = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    t = dict(x=r(1, T, D), g=-r(1, T, D).abs(), z=r(1, T, D), h0=r(n, D), dy=r(1, T, D), dh=r(n, D))
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")

    def run():
        d = {k: v.cuda() for k, v in t.items()}
        y, h, marks = sdm.glr_forward(d["x"], d["g"], d["z"], act="sigmoid", initial_state=d["h0"], cu_seqlens=c)
        dx, dg, dz, dh0 = sdm.glr_backward(d["x"], d["g"], d["z"], d["dy"], marks, act="sigmoid", initial_state=d["h0"], dfinal_state=d["dh"], cu_seqlens=c)
        return {"y": y, "dx": dx, "dg": dg, "dz": dz}, h, dh0

    want, h, dh0 = run()
    t["g"][0, at, 2] = value
    got, hh, ddh0 = run()
    other = [0, 1, 3, 4, 5]
    for k in got:
        assert torch.equal(got[k][..., other], want[k][..., other]), k
        if lens:
            assert torch.equal(got[k][:, 900:], want[k][:, 900:]), k
    assert torch.equal(hh[:, other], h[:, other]) and torch.equal(ddh0[:, other], dh0[:, other])
    end = 900 if lens else T
    # to within roundings: a channel's sums are joined the same way wherever its gates are of one kind
    assert torch.equal(got["y"][:, :at, 2], want["y"][:, :at, 2]) and not torch.isfinite(got["y"][0, at:end, 2]).any()
    assert torch.equal(got["dx"][:, at:, 2], want["dx"][:, at:, 2]) and not torch.isfinite(got["dx"][0, :at, 2]).any()
