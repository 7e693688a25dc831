"""GPU tests of the gated delta rule against the recurrence in 64 bits (tests/delta_ref.py).

Tolerances, set before the first run. Every product and sum is float32's (2^-24 a rounding); a value is the end of
sums of at most dk or dv terms over a state and 64 over a chunk, through the triangular system and back, so its error
is below (dk + dv + 4 * 64) * 2^-24 of the largest magnitude that goes into it, taken as the largest value of the
output (for dg, whose terms cancel, the chunk's sum of |q dq| + |k dk|), plus half a step of the output's type. Long
sequences add nothing that grows: with |k| = 1, beta < 1 and g <= 0 each step shrinks the error it receives."""

import pytest
import torch

from tests import delta_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(B, T, Hk, Hv, dk, dv, ty, seed=0, nseq=None):
    gen = torch.Generator().manual_seed(seed + 1000 * T + dk)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k = rnd(B, T, Hk, dk), rnd(B, T, Hk, dk)
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    n = B if nseq is None else nseq
    return dict(q=q.to(ty), k=k.to(ty), v=rnd(B, T, Hv, dv).to(ty), g=-torch.nn.functional.softplus(rnd(B, T, Hv) - 2),
                beta=torch.sigmoid(rnd(B, T, Hv)), s0=0.3 * rnd(n, Hv, dk, dv), do=rnd(B, T, Hv, dv).to(ty),
                ds=0.3 * rnd(n, Hv, dk, dv))


def near(got, want, terms, name, scale=None):
    got = got.detach().cpu().double()
    want = want.detach()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    eps = torch.finfo(got_type(name)).eps / 2 if isinstance(name, tuple) else 2.0 ** -24
    big = (want.abs().max() if want.numel() else 0.0) if scale is None else scale
    bound = eps * want.abs() + terms * 2.0 ** -24 * big + 1e-30
    off = (got - want).abs()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    assert (off <= bound).all(), f"{name}: off by {float((off / bound).max()):.3g} of the bound"


def got_type(name):
    return name[1]


def dev(d):
    return {k: (t.cuda() if isinstance(t, torch.Tensor) else t) for k, t in d.items()}


def forward(d, sm, **kw):
    import deterministic_fp32_gemm_amd as g
    c = dev(d)
    return g.gdr_forward(c["q"], c["k"], c["v"], c["g"], c["beta"], scale=sm, **{"initial_state": c["s0"], **kw})


def backward(d, sm, **kw):
    import deterministic_fp32_gemm_amd as g
    c = dev(d)
    return g.gdr_backward(c["q"], c["k"], c["v"], c["g"], c["beta"], c["do"], scale=sm,
                          **{"initial_state": c["s0"], "dfinal_state": c["ds"], **kw})


def check_forward(d, ty, sm, cu=None, **kw):
    o, s = forward(d, sm, **kw)
    dk, dv = d["q"].shape[3], d["v"].shape[3]
    wo, ws = R.gdr(d["q"], d["k"], d["v"], d["g"], d["beta"], sm, d["s0"], cu)
    near(o, wo, dk + dv + 256, ("o", ty))
    near(s, ws, dk + dv + 256, "state")


def check_backward(d, ty, sm, cu=None, **kw):
    got = backward(d, sm, **kw)
    want = R.gdr_grads(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], sm, d["s0"], d["ds"], cu)
    n = d["q"].shape[3] + d["v"].shape[3] + 256
    r = d["v"].shape[2] // d["q"].shape[2]
    for x, w, name in zip(got[:3], want[:3], ("dq", "dk", "dv")):
        near(x, w, n, (name, ty))
    terms = sum((a.double().abs() * b.abs()).sum(-1).max() for a, b in ((d["q"], want[0]), (d["k"], want[1]))) * 64
    near(got[3], want[3], n, "dg", float(terms))
    near(got[4], want[4], n * max(1, r), "dbeta", float(want[4].abs().max() + want[1].abs().max()))
    near(got[5], want[5], n, "dstate")


SHAPES = [  # B, T, Hk, Hv, dk, dv
    (1, 1, 1, 1, 1, 1), (2, 1, 2, 4, 64, 64), (1, 2, 1, 3, 17, 33), (1, 63, 2, 2, 64, 16), (2, 64, 1, 2, 128, 64),
    (1, 65, 2, 2, 40, 72), (1, 130, 1, 1, 130, 100), (1, 70, 1, 2, 256, 256), (3, 197, 2, 6, 96, 128), (1, 513, 1, 1, 64, 48),
]


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, ty):
    print("forward", shape, ty, flush=True)
    check_forward(make(*shape, TYPES[ty]), TYPES[ty], shape[4] ** -0.5)


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, ty):
    print("backward", shape, ty, flush=True)
    check_backward(make(*shape, TYPES[ty]), TYPES[ty], shape[4] ** -0.5)


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("shape", [(9, 70, 4, 8, 64, 64), (9, 66, 2, 4, 128, 116)],
                         ids=lambda s: "x".join(map(str, s)))
def test_many_heads(shape, ty):
    """More than 256 slices of 16 state columns: the scans take 32 columns a workgroup."""
    print("many heads", shape, ty, flush=True)
    d = make(*shape, TYPES[ty])
    check_forward(d, TYPES[ty], shape[4] ** -0.5)
    check_backward(d, TYPES[ty], shape[4] ** -0.5)


@pytest.mark.parametrize("ty,dk", [("f32", 24), ("bf16", 72), ("f16", 64)])
def test_shared_heads_of_many_chunks(ty, dk):
    """256 chunks and key heads: one workgroup sums dq and dk over the value heads of a key head."""
    d = make(16, 60, 16, 48, dk, 16, TYPES[ty])
    check_backward(d, TYPES[ty], dk ** -0.5)


def test_packed_sequences():
    """Runs of every awkward length in one row, empty ones first, last and between; the tokens of none get zeros."""
    lens = [0, 1, 64, 0, 63, 65, 130, 2, 0]
    total = sum(lens) + 5           # five tokens of no run
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    cut = torch.tensor(cu, dtype=torch.int32).cuda()
    d = make(1, total, 1, 2, 64, 40, torch.float32, seed=3, nseq=len(lens))
    check_forward(d, torch.float32, 0.125, cu, cu_seqlens=cut)
    check_backward(d, torch.float32, 0.125, cu, cu_seqlens=cut)
    o, s = forward(d, 0.125, cu_seqlens=cut)
    assert not o[:, cu[-1]:].any()
    assert torch.equal(s[0].cpu(), d["s0"][0])      # an empty run's state is the one it came with


@pytest.mark.parametrize("bad", [[0, 300, 100, 400], [-5, 10, 20, 30], [0, 7, 7, 1 << 30]])
def test_bad_runs_stay_in_bounds(bad):
    """Entries that no caller should pass are clamped to the row (the host cannot see them): finite work, and tokens
    of a run that lies within bounds unharmed."""
    d = make(1, 130, 1, 1, 64, 32, torch.float32, nseq=3)
    cut = torch.tensor(bad, dtype=torch.int32).cuda()
    o, s = forward(d, 1.0, cu_seqlens=cut)
    grads = backward(d, 1.0, cu_seqlens=cut)
    torch.cuda.synchronize()
    assert o.shape == (1, 130, 1, 32) and s.shape == (3, 1, 64, 32) and len(grads) == 6


@pytest.mark.parametrize("ty", TYPES)
def test_no_states(ty):
    d = make(2, 90, 2, 2, 32, 24, TYPES[ty])
    z = torch.zeros_like(d["s0"])
    a, _ = forward(d, 0.2, initial_state=None)
    b, s = forward(d, 0.2, initial_state=z.cuda(), final_state=False)
    assert s is None and torch.equal(a, b)
    x = backward(d, 0.2, initial_state=None, dfinal_state=None)
    y = backward(d, 0.2, initial_state=z.cuda(), dfinal_state=z.cuda())
    for p, q in zip(x, y):
        assert torch.equal(p, q)


def test_forgetting():
    """Log decays of -inf (a reset), -200 and 0, beta of 0 and 1: the tokens after a reset keep full accuracy."""
    d = make(1, 150, 1, 2, 48, 32, torch.float32)
    d["g"][0, 20] = -float("inf")
    d["g"][0, 70] = -200.0
    d["g"][0, 100:110] = 0.0
    d["g"][0, 128:140] = -90.0
    d["beta"][0, 30] = 0.0
    d["beta"][0, 31] = 1.0
    check_forward(d, torch.float32, 0.3)
    got = backward(d, 0.3)
    safe = {**d, "g": d["g"].clamp(min=-1000.0)}      # automatic differentiation of exp(-inf) * 0 is NaN
    want = R.gdr_grads(safe["q"], safe["k"], safe["v"], safe["g"], safe["beta"], safe["do"], 0.3, safe["s0"], safe["ds"])
    for x, w, name in zip(got, want, ("dq", "dk", "dv", "dg", "dbeta", "dstate")):
        near(x, w, 4 * (48 + 32 + 256), name)


def test_repeated_keys():
    """One key for all tokens, beta 1, no decay: powers of the triangular system would reach 10^17."""
    d = make(1, 128, 1, 1, 64, 32, torch.float32)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 1.0
    d["g"][:] = 0.0
    check_forward(d, torch.float32, 1.0)


def test_strides():
    """q, k, v as slices of one projection, head-major tensors, shared (expanded) decays, odd alignment."""
    B, T, H, dk, dv = 2, 77, 2, 64, 64
    d = make(B, T, H, H, dk, dv, torch.bfloat16)
    want_o, want_s = forward(d, 0.125)
    want_g = backward(d, 0.125)
    flat = torch.cat([d[x].reshape(B, T, H * 64) for x in "qkv"], -1).cuda()
    q, k, v = (flat[..., i * H * 64:(i + 1) * H * 64].unflatten(-1, (H, 64)) for i in range(3))
    e = {**d, "q": q, "k": k, "v": v}
    odd = torch.empty(d["do"].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(d["do"].shape)
    odd.copy_(d["do"])
    f = {**e, "do": odd, "g": d["g"].cuda().transpose(1, 2).contiguous().transpose(1, 2)}
    major = {**f, "v": v.transpose(1, 2).contiguous().transpose(1, 2)}
    last = {**f, "q": q.transpose(2, 3).contiguous().transpose(2, 3)}       # its last axis is not contiguous
    for x in (e, f, major, last):
        o, s = forward(x, 0.125)
        assert torch.equal(o, want_o) and torch.equal(s, want_s)
        for a, b in zip(backward(x, 0.125), want_g):
            assert torch.equal(a, b)
    one = {**d, "beta": torch.full((1, 1, 1), 0.5).expand(B, T, H)}
    two = {**d, "beta": torch.full((B, T, H), 0.5)}
    assert torch.equal(forward(one, 0.125)[0], forward(two, 0.125)[0])


def test_same_bits_and_other_stream():
    d = make(2, 300, 2, 6, 128, 128, torch.bfloat16)
    o, s = forward(d, 0.1)
    grads = backward(d, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, s2 = forward(d, 0.1)
        grads2 = backward(d, 0.1)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, s2)
    for a, b in zip(grads, grads2):
        assert torch.equal(a, b)


def test_graph():
    """A captured forward and backward, replayed on new inputs with eager calls between."""
    import deterministic_fp32_gemm_amd as g
    ds = [dev(make(1, 140, 1, 2, 64, 64, torch.bfloat16, seed=i)) for i in range(3)]
    names = ("q", "k", "v", "g", "beta", "s0", "do", "ds")
    buf = {n: ds[0][n].clone() for n in names}

    def both(d):
        o, s = g.gdr_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=d["s0"])
        return o, s, *g.gdr_backward(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], initial_state=d["s0"],
                                     dfinal_state=d["ds"])

    want = [both(d) for d in ds]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(buf)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(buf)
    for d, w in list(zip(ds, want)) * 2:
        for n in names:
            buf[n].copy_(d[n])
        graph.replay()
        both(d)
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)


def test_differences():
    """Gradients against differences of the forward itself along random directions, in float32."""
    d = make(1, 100, 1, 2, 32, 32, torch.float32)
    grads = backward(d, 0.25)
    gen = torch.Generator().manual_seed(9)
    names = ("q", "k", "v", "g", "beta", "s0")
    h = 2e-3

    def loss(e):
        o, s = forward(e, 0.25, initial_state=e["s0"].cuda())
        return float((o.double() * d["do"].cuda().double()).sum() + (s.double() * d["ds"].cuda().double()).sum())

    for n, gr in zip(names, grads):
        way = torch.randn(d[n].shape, generator=gen)
        way /= way.norm()
        slope = (loss({**d, n: d[n] + h * way}) - loss({**d, n: d[n] - h * way})) / (2 * h)
        want = float((gr.cpu().double() * way.double()).sum())
        # the loss's own rounding, 2^-24 of sums of thousands of terms of size 1, over 2 h; and h^2 of its curvature
        assert abs(slope - want) <= 2e-2 + 1e-3 * abs(want), (n, slope, want)


# ---- the recurrent form ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1, 1), (3, 1, 2, 4, 64, 64), (2, 3, 1, 3, 40, 72), (5, 1, 2, 2, 130, 33),
                                   (2, 2, 1, 1, 256, 256), (300, 1, 2, 4, 128, 128), (70, 2, 4, 16, 100, 130),
                                   (40, 1, 8, 32, 200, 256)],
                         ids=lambda s: "x".join(map(str, s)))
def test_step(shape, ty):
    import deterministic_fp32_gemm_amd as g
    print("step", shape, ty, flush=True)
    B, T, Hk, Hv, dk, dv = shape
    d = make(*shape, TYPES[ty])
    pool = B + 3
    gen = torch.Generator().manual_seed(1)
    state = 0.3 * torch.randn(pool, Hv, dk, dv, generator=gen)
    slots = torch.randperm(pool, generator=gen)[:B].to(torch.int32)
    idle = torch.zeros(B, dtype=torch.bool)
    if B > 1:
        slots[1], idle[1] = -1, True
    if B > 2:
        slots[2], idle[2] = pool, True
    c = dev(d)
    st = state.cuda()
    o = g.gdr_step(c["q"], c["k"], c["v"], c["g"], c["beta"], st, slots=slots.cuda(), scale=0.2)
    live = [b for b in range(B) if not idle[b]]
    at = slots[live].long()
    wo, ws = R.gdr(*(d[n][live] for n in ("q", "k", "v", "g", "beta")), 0.2, state[at])
    near(o.cpu()[live], wo, dk + 8, ("o", TYPES[ty]))
    near(st.cpu()[at], ws, dk + 8, "state")
    assert not o.cpu()[idle].any()
    rest = torch.ones(pool, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(st.cpu()[rest], state[rest])


def test_step_follows_forward():
    """A prompt by the chunked form, then tokens one by one, against the whole by the chunked form."""
    import deterministic_fp32_gemm_amd as g
    d = dev(make(2, 100, 2, 4, 64, 64, torch.float32))
    sl = lambda a, b: [d[n][:, a:b] for n in ("q", "k", "v", "g", "beta")]  # noqa: E731
    whole, last = g.gdr_forward(*sl(0, 100), initial_state=d["s0"])
    _, state = g.gdr_forward(*sl(0, 90), initial_state=d["s0"])
    for t in range(90, 100):
        out = torch.empty(2, 1, 4, 64, device="cuda")
        o = g.gdr_step(*sl(t, t + 1), state, out=out)
        assert o is out
        near(o.cpu(), whole[:, t:t + 1].cpu().double(), 2 * (64 + 64 + 256), "o")
    near(state.cpu(), last.cpu().double(), 2 * (64 + 64 + 256), "state")


def test_step_wide_offsets():
    """States past the reach of 32-bit element offsets: the last slot of a pool of over 2^31 elements."""
    import deterministic_fp32_gemm_amd as g
    Hv, dk, dv = 32, 128, 128
    pool = (1 << 31) // (Hv * dk * dv) + 2
    state = torch.zeros(pool, Hv, dk, dv, device="cuda")
    d = make(1, 1, Hv, Hv, dk, dv, torch.float32)
    state[-1] = d["s0"][0].cuda()
    c = dev(d)
    o = g.gdr_step(c["q"], c["k"], c["v"], c["g"], c["beta"], state, slots=torch.tensor([pool - 1], dtype=torch.int32).cuda(),
                   scale=1.0)
    wo, ws = R.gdr(d["q"], d["k"], d["v"], d["g"], d["beta"], 1.0, d["s0"])
    near(o.cpu(), wo, dk + 8, "o")
    near(state[-1:].cpu(), ws, dk + 8, "state")
    assert not state[0].any() and not state[-2].any()


def test_stream_argument():
    """A call on a named stream that waits behind other work, while the current stream allocates and writes."""
    import deterministic_fp32_gemm_amd as g
    d = dev(make(2, 300, 2, 6, 128, 128, torch.bfloat16))
    x = [d[n] for n in ("q", "k", "v", "g", "beta")]
    o, s = g.gdr_forward(*x, initial_state=d["s0"])
    want = [o, s, *g.gdr_backward(*x, d["do"], initial_state=d["s0"])]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = [*g.gdr_forward(*x, initial_state=d["s0"], stream=stream),
               *g.gdr_backward(*x, d["do"], initial_state=d["s0"], stream=stream)]
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (2 ** 20, 2 ** 22, 2 ** 24, 2 ** 25) * 3]
        torch.cuda.synchronize()
        del junk
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_scale_is_a_value():
    """A scale held by a tensor is read at every call."""
    import deterministic_fp32_gemm_amd as g
    d = dev(make(1, 30, 1, 1, 32, 32, torch.float32))
    x = [d[n] for n in ("q", "k", "v", "g", "beta")]
    scale = torch.tensor(0.5)
    one = g.gdr_forward(*x, scale=scale)[0]
    scale.fill_(1.0)
    assert torch.equal(g.gdr_forward(*x, scale=scale)[0], 2 * one)
