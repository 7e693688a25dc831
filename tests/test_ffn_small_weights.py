"""The 16-bit feed-forward gradient of small weights and many rows: few values of dWg and dWu, whose error would show what dg and du
lost by their rounding, come from dg and du in two parts.

Bound, element by element and set before the first run. With s the exact value and s' = s + d what is rounded at the end, the result
is the value of the type nearest to s', so it is within |round(s) - s| + 2 |d| of s. d: g and u are given in float32, dg and du have
three operations and a gate, (8 + 16 (1 + |g|)) 2^-24 of |dh u| and |dh|; two parts leave half a step squared of them; and the sum,
of 16 products at a time, rounds or cuts once for each 16 and each of two parts, and 40 times for what joins it, by 2^-23 of the sum of
absolute values."""

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from tests.block_ref import TYPES, act64, half, tiny
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,F", [(200, 40, 40), (110, 60, 50), (600, 16, 16), (400, 8, 64), (400, 64, 8)])
@pytest.mark.parametrize("ty,act", [("bf16", "none"), ("f16", "silu"), ("bf16", "gelu")])
def test_two_parts(ty, act, M, K, F):
    say("ffn small weights", ty, act, M, K, F)
    t = TYPES[ty]
    gen = torch.Generator().manual_seed(M + K)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, wg, wu, dh = r(M, K).to(t), (r(F, K) * K ** -0.5).to(t), (r(F, K) * K ** -0.5).to(t), r(M, F).to(t)
    g, u = (x.float() @ wg.float().t()), (x.float() @ wu.float().t())
    got = sdm.ffn_backward(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), (g.cuda(), u.cuda()), act=act)
    X, G, W, DH, g, u = (v.double() for v in (x, wg, wu, dh, g, u))
    f, df, _ = act64(g, act)
    dg, du = DH * u * df, DH * f
    gate = (8 + 16 * (1 + g.abs())) * 2.0 ** -24
    edg = half(t) ** 2 * dg.abs() + gate * (DH * u).abs() + tiny(t)
    edu = half(t) ** 2 * du.abs() + gate * DH.abs() + tiny(t)
    eps = lambda n: (2 * n / 16 + 40) * 2.0 ** -23  # noqa: E731
    for have, (s, d) in zip(got, (
            (dg @ G + du @ W, edg @ G.abs() + edu @ W.abs() + eps(2 * F) * (dg.abs() @ G.abs() + du.abs() @ W.abs())),
            (dg.t() @ X, edg.t() @ X.abs() + eps(M) * (dg.abs().t() @ X.abs())),
            (du.t() @ X, edu.t() @ X.abs() + eps(M) * (du.abs().t() @ X.abs())))):
        off = (have.double().cpu() - s).abs()
        bound = (s.to(t).double() - s).abs() + 2 * d
        assert (off <= bound).all(), f"{int((off > bound).sum())} of {off.numel()}, by up to {float((off / bound).max()):.3g} times the bound"
