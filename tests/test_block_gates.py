"""The gates of the recurrence and of the feed-forward product far from zero, element by element, where the sigmoid or its
complement is tiny or has left float32.

Each case makes one gated value a product of few factors, so that its error is the gate's. Bounds, set before the first run,
relative to the element: the exponential's argument is rounded once, |z| 2^-24 of its result, two products and a sum double
that at the most; the hardware's functions and the other products are below 64 roundings of 2^-24; then half a step of the type.
Beside that the sigmoid, or 1 minus it, may be zero below 2^-126, which |z| <= 104 then multiplies (from 104 on it is zero in
float32 anyway), and a result below the type's range rounds to a multiple of its smallest step. No part of the bound grows with
|z| where the value does not."""

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from tests.block_ref import TYPES, half, tiny
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

FAR = [-81.0, -85.0, -88.0, -100.0, -104.0, -1e4, -1e30, -1e34, -1e36, -3e38]


def values(t):
    """Gates from -60 to 60, and far ones of either sign, as far as four times act(z) is in the type."""
    far = torch.tensor(FAR + [-v for v in FAR] + [0.0, -1.0, 1.0]).clamp(torch.finfo(t).min, torch.finfo(t).max / 4)
    return torch.cat([torch.linspace(-60, 60, 101), far]).to(t)


def gate(z, act):
    """act and act' in 64 bits, without a difference of nearly equal numbers."""
    e = torch.exp(-z.abs())
    small, large = e / (1 + e), 1 / (1 + e)
    p, q = torch.where(z < 0, small, large), torch.where(z < 0, large, small)
    return (p, p * q) if act == "sigmoid" else (torch.where(p == 0, 0.0, z * p), torch.where(p == 0, 0.0, p * (1 + z * q)))


def near(got, by, z, act, ty, what):
    """got against by * act(z) or by * act'(z)"""
    a, d = gate(z, act)
    want = by * (a if what == "value" else d)
    off = (got.double().cpu() - want).abs()
    bound = (2 * z.abs().clamp(max=110) + 64) * 2.0 ** -24 * want.abs() + half(ty) * want.abs() + 104 * 2.0 ** -126 * by.abs() + tiny(ty)
    if act == "silu" and what != "value":       # 1 + z (1 - p) crosses zero near z = -1.28
        bound = bound + 64 * 2.0 ** -24 * by.abs() * (z.abs() < 4)
    assert (off <= bound).all(), f"{what}: at z = {z[(off > bound)][:4].tolist()}: {got.flatten()[(off > bound).flatten().to(got.device)][:4].tolist()}"


@pytest.mark.parametrize("T", [1, 5, 140, 1300])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("ty", TYPES)
def test_recurrence(ty, act, T):
    """Every token forgets the others: y = x act(z), dz = dy x act'(z); walked runs, several tiles and tiles from the queue."""
    say("gate glr", ty, act, T)
    t = TYPES[ty]
    z = values(t)
    z = z.repeat(T, 1)[None].contiguous()
    gen = torch.Generator().manual_seed(T)
    x, dy = ((0.5 + torch.rand(z.shape, generator=gen)).to(t) for _ in range(2))
    g = torch.full(z.shape, -float("inf"))
    X, G, Z, DY = (v.cuda() for v in (x, g, z, dy))
    y, _, marks = sdm.glr_forward(X, G, Z, act=act)
    near(y, x.double(), z.double(), act, t, "value")
    dx, _, dz, _ = sdm.glr_backward(X, G, Z, DY, marks, act=act)
    near(dx, dy.double(), z.double(), act, t, "value")
    near(dz, dy.double() * x.double(), z.double(), act, t, "derivative")
    if T <= 5:
        near(sdm.glr_step(X, G, Z, torch.zeros(1, z.shape[2], device="cuda"), act=act), x.double(), z.double(), act, t, "value")


@pytest.mark.parametrize("M", [3, 70, 300])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("ty", TYPES)
def test_product(ty, act, M):
    """One value a row and a weight of it: g = x wg is exact, u = 1 for x = 1; then dwu = sum dh act(g) of one row that has any."""
    say("gate ffn", ty, act, M)
    t = TYPES[ty]
    z = values(t)
    one = torch.ones(M, 1, dtype=t)
    wg, wu = z[:, None].contiguous(), torch.ones(len(z), 1, dtype=t)
    X, WG, WU = (v.cuda() for v in (one, wg, wu))
    h, kept = sdm.ffn_forward(X, WG, WU, act=act, keep=True)
    every = z.double().expand(M, -1)
    assert torch.equal(kept[0].cpu(), z.float().expand(M, -1)) and (kept[1] == 1).all()
    near(h, torch.ones_like(every), every, act, t, "value")
    # dwg = dg^T x: dg = dh act'(g) where dh is not zero, one row; the rounding to the type twice at the most
    dh = torch.zeros(M, len(z), dtype=t)
    dh[M // 2] = 1.5
    _, dwg, dwu = sdm.ffn_backward(dh.cuda(), X, WG, WU, kept, act=act)
    by = torch.full((len(z),), 1.5, dtype=torch.float64)
    near(dwg[:, 0], by, z.double(), act, t, "derivative")
    near(dwu[:, 0], by, z.double(), act, t, "value")


def test_product_in_8_bits():
    z = torch.tensor(FAR + [-v for v in FAR] + [-20.0, 20.0])
    q, s = sdm.quant_rows(z[:, None].cuda())
    q1, s1 = sdm.quant_rows(torch.ones(len(z), 1).cuda())
    for M in (3, 70):
        x, sx = sdm.quant_rows(torch.ones(M, 1).cuda())
        for act in ("sigmoid", "silu"):
            h, kept = sdm.ffn_forward(x, q, q1, act=act, x_scale=sx, gate_scale=s, up_scale=s1, keep=True)
            near(h / kept[1].to(h.dtype), torch.ones(M, len(z), dtype=torch.float64), kept[0].double().cpu(), act, torch.bfloat16, "value")


def test_infinite_gates():
    """sigmoid is 0 and 1 there; z sigmoid(z) at -inf is -inf times 0."""
    inf = float("inf")
    for ty in TYPES.values():
        z = torch.tensor([[[-inf, inf]]], dtype=ty, device="cuda")
        x = torch.full_like(z, 2.0)
        assert sdm.glr_forward(x, x, z, act="sigmoid")[0].flatten().tolist() == [0.0, 2.0]
        y = sdm.glr_forward(x, x, z, act="silu")[0].flatten()
        assert torch.isnan(y[0]) and y[1] == inf
