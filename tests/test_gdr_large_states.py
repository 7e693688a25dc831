"""GPU tests of 16-bit outputs that cancel against large states: a key that overwrites what the state holds leaves
o = scale S^T q, where scale exp(G) Q S and P U are each as large as the state and their sum is as small as v.

Tolerances, set before the first run. With one unit vector a token as q and k, beta 1 and g 0, o is scale v exactly and
every step but these is exact in float32 (scale a power of two, the triangular matrix the identity): U = v - S, one
rounding, and the sum of o's parts, at most 12 products in two accumulators and their sum; 32 steps of 2^-24 of
scale (|S| + |v|) hold them all, and half a step of the output's type the last. With q and k of any direction the bound
is that of test_gdr.py."""

import pytest
import torch

from tests import delta_ref as R
from tests import test_gdr as G

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("size", [30.0, 1000.0, 30000.0])
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("shape", [(1, 40, 1, 2, 64, 48), (1, 100, 1, 1, 128, 64), (1, 70, 2, 2, 256, 40),
                                   (9, 50, 4, 8, 64, 64), (9, 66, 2, 4, 128, 116)], ids=lambda s: "x".join(map(str, s)))
def test_overwritten_rows(shape, ty, size):
    print("overwritten", shape, ty, size, flush=True)
    B, T, Hk, Hv, dk, dv = shape
    d = G.make(*shape, TYPES[ty])
    unit = torch.eye(dk)[:T].expand(Hk, T, dk).transpose(0, 1).expand(B, T, Hk, dk).contiguous()
    d["q"] = d["k"] = unit.to(TYPES[ty])
    d["g"], d["beta"] = torch.zeros(B, T, Hv), torch.ones(B, T, Hv)
    gen = torch.Generator().manual_seed(T)
    d["s0"] = size * (0.5 + 0.5 * torch.rand(B, Hv, dk, dv, generator=gen)) * torch.randn(B, Hv, dk, dv, generator=gen).sign()
    o, s = G.forward(d, 0.125)
    v = d["v"].double()
    want = 0.125 * v
    bound = torch.finfo(TYPES[ty]).eps / 2 * want.abs() + 32 * 2.0 ** -24 * 0.125 * (size + v.abs().max())
    off = (o.cpu().double() - want).abs()
    assert (off <= bound).all(), f"o: off by {float((off / bound).max()):.3g} of the bound"
    rows = v.transpose(1, 2)        # the state's first T rows are v, the others what they were
    off = (s[:, :, :T].cpu().double() - rows).abs()
    assert (off <= 32 * 2.0 ** -24 * (size + v.abs().max())).all()
    assert torch.equal(s[:, :, T:].cpu(), d["s0"][:, :, T:])


@pytest.mark.parametrize("size", [30.0, 100.0])
@pytest.mark.parametrize("ty", TYPES)
def test_any_direction(ty, size):
    print("any direction", ty, size, flush=True)
    d = G.make(1, 64, 1, 1, 64, 64, TYPES[ty])
    d["q"] = d["k"]
    d["beta"] = torch.ones(1, 64, 1)
    d["s0"] = d["s0"] * (size / 0.3)
    o, _ = G.forward(d, 0.125)
    wo, _ = R.gdr(d["q"], d["k"], d["v"], d["g"], d["beta"], 0.125, d["s0"])
    G.near(o, wo, 64 + 64 + 256, ("o", TYPES[ty]))
