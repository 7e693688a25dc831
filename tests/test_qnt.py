"""Rows in 8 bits on the GPU against their definition in 64 bits."""

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from tests.block_ref import TYPES, U, e4m3_step
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def inputs(ty, rows, D, res, wty=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (r(rows, D) * torch.exp(2 * r(rows, 1))).to(TYPES[ty]).cuda()
    return x, r(rows, D).to(TYPES[ty]).cuda() if res else None, (1 + 0.3 * r(D)).to(TYPES[wty or ty]).cuda()


def check(q, scale, y):
    """q and scale of rows whose values are y in 64 bits. The mean is a sum of D squares in a tree of some 40 roundings at the
    deepest, under a root: 24 roundings; y and the division by the scale have 5 more."""
    assert q.dtype == torch.float8_e4m3fn and scale.dtype == torch.float32
    want = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    assert ((scale.double() - want).abs() <= 32 * U * want).all()
    v, at = q.double(), y / scale.double()[..., None]
    assert ((v - at).abs() <= 0.5 * e4m3_step(at) + 64 * U * at.abs()).all()


def reference(x, w, eps=1e-6):
    X = x.double()
    return X * torch.rsqrt(X.square().mean(-1, keepdim=True) + eps) * w.double()


@pytest.mark.parametrize("ty,wty,rows,D,res", [
    ("f32", None, 1, 1, True), ("f32", None, 9, 7, True), ("bf16", None, 3, 8, False), ("f16", "f32", 70, 100, True),
    ("bf16", "f32", 5, 512, True), ("f32", None, 5, 513, False), ("bf16", None, 16, 2048, True), ("f16", None, 3, 2049, True),
    ("bf16", None, 33, 4096, True), ("f32", None, 3, 4097, True), ("bf16", None, 7, 8192, True), ("f32", None, 2, 8193, True),
    ("f16", None, 2, 16383, True), ("f32", None, 2, 16384, False), ("bf16", None, 20000, 129, True),
])
def test_norm_quant(ty, wty, rows, D, res):
    say("norm_quant", ty, wty, rows, D, res)
    x, r, w = inputs(ty, rows, D, res, wty)
    q, scale, xn = sdm.norm_quant(x, r, w)
    if res:
        assert torch.equal(xn, (x.float() + r.float()).to(x.dtype))
    else:
        assert xn is x
    check(q, scale, reference(xn, w))


@pytest.mark.parametrize("ty,rows,D", [("f32", 1, 1), ("f16", 5, 7), ("bf16", 40, 300), ("f32", 3, 3001), ("bf16", 2, 16384)])
def test_quant_rows(ty, rows, D):
    say("quant_rows", ty, rows, D)
    x = inputs(ty, rows, D, False)[0]
    q, scale = sdm.quant_rows(x)
    check(q, scale, x.double())
    # the largest of a row stands for itself
    top = x.double().abs().amax(-1)
    assert ((q.double().abs().amax(-1) * scale.double() - top).abs() <= 2 * U * top).all()


def test_rows_of_zeros_and_tiny_values():
    x = torch.zeros(3, 40, device="cuda")
    x[1] = 1e-42
    x[2, 5] = -3.0
    q, scale = sdm.quant_rows(x)
    assert (scale[:2] == 2.0 ** -126).all() and not q[0].double().any()
    assert ((q[1].double() * scale[1].double() - x[1].double()).abs() <= 2.0 ** -10 * 2.0 ** -126).all()
    assert q[2, 5].double() == -448 and not q[2, :5].double().any()
    q, scale, _ = sdm.norm_quant(x[:1], None, torch.ones(40, device="cuda"))
    assert scale[0] == 2.0 ** -126 and not q.double().any()


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_a_value_that_is_not_finite_spoils_its_row_alone(value):
    x, r, w = inputs("f32", 5, 700, True)
    want = sdm.norm_quant(x, r, w)
    x[2, 699] = value
    q, scale, xn = sdm.norm_quant(x, r, w)
    keep = [0, 1, 3, 4]
    assert torch.equal(q[keep].view(torch.uint8), want[0][keep].view(torch.uint8)) and torch.equal(scale[keep], want[1][keep])
    assert torch.isnan(scale[2]) and torch.isnan(q[2].float()).all()
    q, scale = sdm.quant_rows(x)
    assert torch.isnan(scale[2]) and torch.isnan(q[2].float()).all() and torch.isfinite(scale[keep]).all()


def test_a_mean_beyond_float32_spoils_its_row():
    x = torch.full((2, 64), 1.0, device="cuda")
    x[1] = 1e30
    q, scale, _ = sdm.norm_quant(x, None, torch.ones(64, device="cuda"))
    assert torch.isfinite(scale[0]) and torch.isnan(scale[1]) and torch.isnan(q[1].float()).all()
    q, scale = sdm.quant_rows(x)
    assert torch.isfinite(scale).all() and (q[1].float() == 448).all()


def test_shapes_strides_and_empty():
    x, r, w = inputs("bf16", 12, 50, True)
    want = sdm.norm_quant(x, r, w)
    wide = torch.zeros(12, 103, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:53], wide[:, 53:] = x, r
    got = sdm.norm_quant(wide[:, 3:53], wide[:, 53:], w)
    cols = sdm.norm_quant(x.t().contiguous().t(), r, torch.stack([w, w], 1)[:, 0])
    deep = sdm.norm_quant(x.view(3, 4, 50), r.view(3, 4, 50), w)
    assert deep[0].shape == (3, 4, 50) and deep[1].shape == (3, 4)
    for a in (got, cols, tuple(t.reshape(s.shape) for t, s in zip(deep, want))):
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, want))
    q, scale, xn = sdm.norm_quant(x[:0], r[:0], w)
    assert q.shape == (0, 50) and scale.shape == (0,) and xn.shape == (0, 50)


def test_graph_and_stream():
    x, r, w = inputs("bf16", 300, 700, True)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = sdm.norm_quant(x, r, w, stream=side)
    torch.cuda.synchronize()
    want = sdm.norm_quant(x, r, w)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(on_side, want))
    with torch.cuda.graph(graph):
        got = sdm.norm_quant(x, r, w)
    for seed in range(1, 4):
        x.copy_(inputs("bf16", 300, 700, True, seed=seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, sdm.norm_quant(x, r, w)))


def test_no_gradient():
    x, r, w = inputs("f32", 4, 20, True)
    w.requires_grad_()
    q, scale, xn = sdm.norm_quant(x, r, w)
    for t in (scale, xn):
        with pytest.raises(RuntimeError, match="norm_quant has no gradient"):
            t.sum().backward(retain_graph=True)
