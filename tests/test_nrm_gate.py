"""GPU tests of the block norm's gate far from zero, where act'(z) is tiny on one side, element by element.

Without a second norm dz = dx_new scale o r1 w_post act'(z), one product chain an element. Tolerances, set before the first
run, relative to the element: the exponential's argument is rounded once, |z| 2^-24 of its result, and squares and sums of
it double that; the row's norm, two hardware functions and the products are below 64 roundings of 2^-24; then half a step
of the type (of its subnormals, for float16)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def gate(z, act):
    """act and act' in 64 bits, without a difference of nearly equal numbers."""
    small, large = torch.exp(-z.abs()) / (1 + torch.exp(-z.abs())), 1 / (1 + torch.exp(-z.abs()))
    p, q = torch.where(z < 0, small, large), torch.where(z < 0, large, small)
    return (p, p * q) if act == "sigmoid" else (z * p, p * (1 + z * q))


@pytest.mark.parametrize("D", [96, 1111, 4608])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("ty", TYPES)
def test_far_gates(ty, act, D):
    import deterministic_fp32_gemm_amd as g
    print("gate", ty, act, D, flush=True)
    t = TYPES[ty]
    gen = torch.Generator().manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    rows = 5
    z = (torch.rand(rows, D, generator=gen) * 60 - 30).to(t)
    z[0] = z[0].abs().clamp(min=8)
    z[1] = -z[1].abs().clamp(min=8)
    o = (r(rows, D).sign() * (0.5 + torch.rand(rows, D, generator=gen))).to(t)
    dx = (r(rows, D).sign() * (0.5 + torch.rand(rows, D, generator=gen))).to(t)
    w, scale = (1 + 0.2 * torch.rand(D, generator=gen) for _ in range(2))
    c = [x.cuda() for x in (o, z, w, scale)]
    xn, _, rstd = g.norm_forward(None, *c[:3], None, c[3], act=act, eps=1e-6)
    got = g.norm_backward(dx.cuda(), None, None, *c[:3], None, c[3], rstd, act=act)
    o, z, dx, w, scale = (x.double() for x in (o, z, dx, w, scale))
    n = o / (o.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    a, d = gate(z, act)
    eps, least = torch.finfo(t).eps / 2, 2.0 ** -25 if ty == "f16" else 2.0 ** -134 if ty == "bf16" else 2.0 ** -126
    for have, want, name in ((got[2], dx * scale * n * w * d, "dz"), (xn, scale * n * w * a, "x_new")):
        off = (have.cpu().double() - want).abs()
        bound = ((2 * z.abs() + 64) * 2.0 ** -24 + eps) * want.abs() + least
        if act == "silu" and name == "dz":      # 1 + z (1 - p) crosses zero near z = -1.28
            bound = bound + 64 * 2.0 ** -24 * (dx * scale * n * w).abs() * (z.abs() < 4)
        assert (off <= bound).all(), f"{name}: off by {float((off / bound).max()):.3g} of the bound"
