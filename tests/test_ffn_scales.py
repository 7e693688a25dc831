"""The gated feed-forward product of 8-bit rows whose scales' product leaves float32 while the products themselves do not. Few rows
and tiles; the bounds are those of tests/block_ref.py."""

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from tests.block_ref import ffn, within
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("M", [3, 70, 300])
@pytest.mark.parametrize("sx,sw,value", [(1e-24, 1e-20, 448.0), (2.0 ** -126, 2.0 ** -20, 448.0), (2e30, 1e10, 2.0 ** -9), (2e30, 1e10, 0.0),
                                         (1e37, 1e-37, 0.5), (1e-37, 1e37, 0.5), (3.0, 0.7, 8.0)])
def test_scales_far_apart_and_far_from_one(sx, sw, value, M):
    say("ffn scales", sx, sw, value, M)
    K, F = (512 if value == 448 else 32), 40
    x, w = torch.full((M, K), value).to(F8).cuda(), torch.full((F, K), value).to(F8).cuda()
    gen = torch.Generator().manual_seed(M)
    scale = lambda n, s: (s * (1 + torch.rand(n, generator=gen))).cuda()  # noqa: E731
    s = scale(M, sx), scale(F, sw), scale(F, sw)
    h, kept = sdm.ffn_forward(x, w, w, act="silu", x_scale=s[0], gate_scale=s[1], up_scale=s[2], keep=True)
    want = ffn(x, w, w, "silu", h.dtype, s)
    for got, name in zip(kept, "gu"):
        assert torch.isfinite(want[name][0]).all() and want[name][0].abs().max() < 3e38
        within(got, *want[name], name)
    if want["h"][0].abs().max() < 3e38:
        within(h, *want["h"], "h")
