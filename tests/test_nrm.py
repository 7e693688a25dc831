"""GPU tests of the block norm against its definition in 64 bits (tests/delta_ref.py).

Tolerances, set before the first run: float32 arithmetic on a row of D values, whose mean square is a sum of D terms
(a tree of at most 64 sequential ones a lane and 20 levels): 128 * 2^-24 of the largest value that goes into an output,
plus half a step of its type. x_new enters y as it is stored, and where its rounding falls differently from the
definition's (float32 against float64 before the rounding) y moves by one step of the type: y has a whole step. Weights'
gradients are float32 sums over the rows of values up to the largest product: rows * 2^-24 of that, at the worst."""

import pytest
import torch

from tests import delta_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
SIZES = [(1, 1), (3, 7), (5, 64), (4, 511), (9, 512), (2, 520), (7, 1111), (3, 2048), (33, 2050), (2, 4096), (5, 4100),
         (2, 8192), (700, 96)]


def make(rows, D, ty, wt, act, seed=0):
    gen = torch.Generator().manual_seed(seed + rows * 10007 + D)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {n: rnd(rows, D).to(ty) for n in ("x", "o", "z", "dy", "dxn")}
    d |= {n: (1 + 0.3 * rnd(D)).to(wt) for n in ("w_post", "w_pre", "scale")}
    if act == "none":
        d["z"] = None
    return d


def cuda(t):
    return None if t is None else t.cuda()


def near(got, want, ty, name, steps=0.5, terms=128, big=None):
    assert (got is None) == (want is None), name
    if got is None:
        return
    assert got.dtype == ty, name
    got = got.cpu().double()
    want = want.detach()
    big = want.abs().max() if big is None else big
    bound = steps * torch.finfo(ty).eps * want.abs() + terms * 2.0 ** -24 * big
    if ty == torch.float16:
        bound = bound + 2.0 ** -25      # half a step of its subnormals
    off = (got - want).abs()
    assert torch.isfinite(got).all() and (off <= bound).all(), f"{name}: off by {float((off / bound).max()):.3g} of the bound"


def forward(d, act):
    import deterministic_fp32_gemm_amd as g
    return g.norm_forward(*(cuda(d[n]) for n in ("x", "o", "z", "w_post", "w_pre", "scale")), act=act, eps=EPS)


def backward(d, act, xn, rstd):
    import deterministic_fp32_gemm_amd as g
    return g.norm_backward(*(cuda(t) for t in (d["dxn"], d["dy"], xn, d["o"], d["z"], d["w_post"], d["w_pre"], d["scale"],
                                               rstd)), act=act)


def check(d, act, ty, wt):
    xn, y, rstd = forward(d, act)
    wx, _, r1, r2 = R.norm(d["x"], d["o"], d["z"], d["w_post"], d["w_pre"], d["scale"], act, EPS, ty)
    if d["o"] is not None:
        near(xn, wx, ty, "x_new")
        near(rstd[:, :1], r1, torch.float32, "r1")
    if d["w_pre"] is not None:
        kept = xn.cpu() if d["o"] is not None else d["x"]      # y is the norm of what was stored
        _, wy, _, r2 = R.norm(kept, None, None, None, d["w_pre"], None, act, EPS, ty)
        near(y, wy, ty, "y")
        near(rstd[:, 1:], r2, torch.float32, "r2")
    kept = xn.cpu() if xn is not None else None
    got = backward(d, act, kept, rstd)
    want = R.norm_grads(d["dxn"], d["dy"], kept, d["o"], d["z"], d["w_post"], d["w_pre"], d["scale"], act, EPS)
    rows = (d["o"] if d["o"] is not None else d["x"]).shape[0]
    peak = float(want[0].abs().max()) * 8 * 4
    for a, b, name in zip(got[:3], want[:3], ("dx", "do", "dz")):
        near(a, b, ty, name, big=None if b is None else b.abs().max() + peak / 32)
    for a, b, name in zip(got[3:], want[3:], ("dw_post", "dw_pre", "dscale")):
        near(a, b, wt, name, terms=rows + 128, big=peak)


@pytest.mark.parametrize("kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")],
                         ids="-".join)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_norm(size, kind):
    print("norm", size, kind, flush=True)
    ty, wt = TYPES[kind[0]], TYPES[kind[1]]
    act = ("silu", "sigmoid", "none")[(size[0] + size[1]) % 3]
    check(make(*size, ty, wt, act), act, ty, wt)


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
def test_parts(act):
    """Without a residual, without the second norm, the second norm alone, without the direct gradient."""
    ty = torch.float32
    d = make(6, 300, ty, ty, act)
    check({**d, "x": None}, act, ty, ty)
    check({**d, "w_pre": None, "dy": None}, act, ty, ty)
    check({**d, "dxn": None}, act, ty, ty)
    if act == "none":
        only = {**d, "o": None, "z": None, "w_post": None, "scale": None}
        check(only, act, ty, ty)
        check({**only, "dxn": None}, act, ty, ty)


def test_strides_and_shapes():
    import deterministic_fp32_gemm_amd as g
    d = make(12, 264, torch.bfloat16, torch.bfloat16, "silu")
    want = forward(d, "silu")
    wide = torch.empty(12, 3 * 264 + 1, dtype=torch.bfloat16, device="cuda")
    x, o, z = (wide[:, i * 264 + 1:(i + 1) * 264 + 1] for i in range(3))       # rows off every 16-byte boundary
    for t, n in ((x, "x"), (o, "o"), (z, "z")):
        t.copy_(d[n])
    w = [d[n].cuda() for n in ("w_post", "w_pre", "scale")]
    got = g.norm_forward(x, o, z, *w, act="silu", eps=EPS)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    three = [d[n].cuda().view(3, 4, 264) for n in ("x", "o", "z")]
    got = g.norm_forward(*three, *w, act="silu", eps=EPS)
    assert got[0].shape == (3, 4, 264) and torch.equal(got[1].view(12, 264), want[1])
    col = d["o"].cuda().t().contiguous().t()        # column-major
    assert torch.equal(g.norm_forward(d["x"].cuda(), col, d["z"].cuda(), *w, act="silu", eps=EPS)[0], want[0])


def test_empty_and_zero_rows():
    import deterministic_fp32_gemm_amd as g
    d = make(1, 40, torch.float32, torch.float32, "silu")
    e = {n: (t[:0] if t is not None and t.dim() == 2 else t) for n, t in d.items()}
    xn, y, rstd = forward(e, "silu")
    assert xn.shape == (0, 40) and y.shape == (0, 40) and rstd.shape == (0, 2)
    grads = backward(e, "silu", xn.cpu(), rstd)
    assert grads[0].shape == (0, 40) and not any(t.any() for t in grads[3:])
    # a row of zeros: the norm is eps's, nothing divides by zero
    z = torch.zeros(2, 40).cuda()
    xn, y, rstd = g.norm_forward(z, z, z, *(d[n].cuda() for n in ("w_post", "w_pre", "scale")), act="silu", eps=EPS)
    assert not xn.any() and not y.any() and torch.isfinite(rstd).all()


def test_values_that_are_not_finite_stay_in_their_row():
    d = make(4, 600, torch.float32, torch.float32, "silu")
    want = forward(d, "silu")
    for bad in (float("inf"), float("nan")):
        e = {**d, "o": d["o"].clone()}
        e["o"][2, 17] = bad
        got = forward(e, "silu")
        for a, b in zip(got, want):
            keep = [0, 1, 3]
            assert torch.equal(a[keep], b[keep]) and not torch.isfinite(a[2]).all()


def test_large_and_tiny_rows():
    """Rows whose squares would leave float16, and bfloat16 rows near 10^15: sums are float32's."""
    for ty, size in ((torch.float16, 3e4), (torch.bfloat16, 1e15), (torch.float32, 1e-12)):
        d = make(3, 500, ty, torch.float32, "none")
        d["o"] = (d["o"].float().clamp(-1, 1) * size).to(ty)
        xn, y, rstd = forward(d, "none")
        wx, _, _, _ = R.norm(d["x"], d["o"], None, d["w_post"], d["w_pre"], d["scale"], "none", EPS, ty)
        near(xn, wx, ty, "x_new")


def test_same_bits():
    d = make(3000, 1024, torch.bfloat16, torch.bfloat16, "silu")
    xn, y, rstd = forward(d, "silu")
    a = backward(d, "silu", xn.cpu(), rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = backward(d, "silu", xn.cpu(), rstd)
    torch.cuda.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_graph():
    import deterministic_fp32_gemm_amd as g
    ds = [{n: t.cuda() for n, t in make(50, 640, torch.bfloat16, torch.float32, "silu", seed=i).items()} for i in range(3)]
    buf = {n: t.clone() for n, t in ds[0].items()}

    def both(d):
        xn, y, rstd = g.norm_forward(d["x"], d["o"], d["z"], d["w_post"], d["w_pre"], d["scale"], act="silu")
        return xn, y, rstd, *g.norm_backward(d["dxn"], d["dy"], xn, d["o"], d["z"], d["w_post"], d["w_pre"], d["scale"],
                                             rstd, act="silu")

    want = [both(d) for d in ds]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(buf)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(buf)
    for d, w in list(zip(ds, want)) * 2:
        for n in buf:
            buf[n].copy_(d[n])
        graph.replay()
        both(d)
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("size,kind", [((2700, 1111), "f32"), ((1700, 2050), "bf16"), ((2100, 4101), "f16"),
                                       ((4200, 601), "bf16"), ((8300, 17), "f32"), ((8200, 5), "f16")],
                         ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else s)
def test_more_rows_than_workgroups(size, kind):
    """Workgroups that take several rows each, of lengths that end inside a thread's eight columns."""
    print("rows", size, kind, flush=True)
    ty = TYPES[kind]
    check(make(*size, ty, ty, "silu"), "silu", ty, ty)
