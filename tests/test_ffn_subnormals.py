"""Operands of the feed-forward product below their type's normal range, few rows and tiles, forward and gradient: they count as they
are. Powers of two and small multiples of them, whose products and sums float32 holds exactly.

More than 32 float32 rows are split into three bfloat16 parts, whose smallest step is 2^-133: what an operand has below it is lost,
2^-134 at the most, and a product's sum is off by that times the other operand's absolute sum."""

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("ty,small", [(torch.float16, 2.0 ** -24), (torch.float16, 2.0 ** -16), (torch.bfloat16, 2.0 ** -133), (torch.float32, 2.0 ** -140), (torch.float32, 2.0 ** -130)])
def test_forward(ty, small, M):
    """x below the range, weights that bring the product back into float32's."""
    say("ffn subnormal", ty, small, M)
    K, F, back = 64, 40, (1.0 if ty == torch.float16 else 2.0 ** 100)
    gen = torch.Generator().manual_seed(M)
    n, m = torch.randint(0, 5, (M, K), generator=gen), torch.randint(-3, 4, (F, K), generator=gen)
    x, w = (n.double() * small).to(ty), (m.double() * back).to(ty)
    want = n.double() @ m.double().t() * small * back
    least = lambda rows: 2.0 ** -134 * w.double().abs().sum(1) if ty == torch.float32 and rows > 32 else torch.zeros(F)  # noqa: E731
    h, kept = sdm.ffn_forward(x.cuda(), w.cuda(), w.cuda(), act="none", keep=True)
    for g in kept:
        assert ((g.double().cpu() - want).abs() <= least(M)).all()
    h, kept = sdm.ffn_forward(w.cuda(), x.cuda(), x.cuda(), act="none", keep=True)
    assert ((kept[0].double().cpu() - want.t()).abs() <= least(F)[:, None]).all()


@pytest.mark.parametrize("M", [3, 300, 900])
@pytest.mark.parametrize("precise", [False, True])
def test_gradient_of_small_values_in_float16(precise, M):
    """dg and du of float16 are below its normal range throughout: dh of 2^-20 and gates of 1 with act none."""
    K, F = 40, 96
    gen = torch.Generator().manual_seed(M)
    r = lambda a, b, *s: torch.randint(a, b, s, generator=gen).double()  # noqa: E731
    x, wg, wu, dh = r(-2, 3, M, K), r(-2, 3, F, K), r(-2, 3, F, K), r(-7, 8, M, F) * 2.0 ** -20
    one = torch.ones(M, F, device="cuda")
    got = sdm.ffn_backward(*(v.half().cuda() for v in (dh, x, wg, wu)), (one, 2 * one), act="none", precise=precise)
    dg, du = 2 * dh, dh
    for v, want in zip(got, (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x)):
        assert torch.equal(v.cpu(), want.half())
