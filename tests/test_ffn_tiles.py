"""Every kernel of the feed-forward product that the host can choose, each element type with each tile in each direction, with sums
in parts and whole: a host test holds the choice for each shape here, a GPU test its results against the definition in 64 bits (the
bounds of tests/block_ref.py). Every shape ends inside a tile, a block and a piece in M, K and F."""

import ctypes

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from tests.block_ref import TYPES, ffn, within
from tests.block_stub import call, library
from tests.gpu_util import say
from tests.test_block_host import ffn as args

KIND = {"bf16": 0, "f16": 1, "e4m3": 2, "f32": 3}          # of the matrix cores' operands
DTYPE = {"f32": 0, "bf16": 1, "f16": 2, "e4m3": 3}

# forward: rows, lengths, weights' rows, and the tile; 0: few rows
FORWARD = [(m, 100, 41, 0) for m in (1, 15, 16)] + [(17, 100, 41, 64), (1100, 90, 1900, 128), (4010, 70, 2010, 256),
                                                           (4200, 70, 2010, 128), (6010, 70, 2010, 256)]
FORWARD_F32 = [(m, 100, 41, 0) for m in (16, 17, 31, 32)] + [(33, 100, 41, 64), (1100, 90, 1900, 128), (4010, 70, 2010, 128)]
# gradient: rows, lengths, weights' rows, the tile, the parts of dx's sums and of the weights'
GRADIENT = [(130, 90, 70, 64, 1, 1), (3, 200, 3001, 64, 21, 1), (4001, 66, 70, 64, 1, 7), (300, 1801, 1003, 128, 1, 1), (100, 1301, 1801, 128, 7, 1),
            (9001, 501, 61, 128, 1, 16), (601, 3501, 2003, 256, 6, 1), (100, 2601, 3003, 256, 11, 1), (9001, 2049, 2001, 256, 1, 1)]
GRADIENT_F32 = [(130, 90, 70, 64, 1, 1), (3, 200, 3001, 64, 21, 1), (3001, 66, 70, 64, 1, 11), (1501, 1701, 501, 128, 1, 1), (100, 1301, 1501, 128, 11, 1),
                (9001, 501, 61, 128, 1, 32), (300, 1801, 1003, 128, 7, 1)]
FORWARDS = [(ty, *s) for ty in ("bf16", "f16", "e4m3") for s in FORWARD] + [("f32", *s) for s in FORWARD_F32]
GRADIENTS = [(ty, *s) for ty in ("bf16", "f16") for s in GRADIENT] + [("f32", *s) for s in GRADIENT_F32]


def struct(ty, M, K, F):
    """Arguments at made-up addresses far enough apart."""
    a = args(dtype=DTYPE[ty], otype=1 if ty == "e4m3" else DTYPE[ty], M=M, K=K, F=F)
    for i, (n, ld) in enumerate((("x", K), ("wg", K), ("wu", K), ("h", F), ("gate", F), ("up", F), ("dh", F), ("dx", K), ("dwg", K), ("dwu", K))):
        setattr(a, n, (i + 1) << 36)
        setattr(a, "ld_" + n, ld)
    if ty == "e4m3":
        a.sx, a.sg, a.su = 20 << 36, 21 << 36, 22 << 36
    return a


def made(name, a, backward):
    n = library().sdm_ffn_workspace(ctypes.byref(a), backward)
    assert n >= 0
    status, notes = call(name, ctypes.byref(a), 30 << 36, n, None)
    assert status == 0
    return {kind: rest for kind, *rest in notes}


@pytest.mark.parametrize("ty,M,K,F,tile", FORWARDS)
def test_forward_choice(ty, M, K, F, tile):
    notes = made("sdm_ffn_forward", struct(ty, M, K, F), 0)
    if tile:
        assert notes["pair"][:2] == [KIND[ty], tile] and "few" not in notes
    else:
        assert notes == {"few": [DTYPE[ty], 0, 0, 0]}


@pytest.mark.parametrize("ty,M,K,F,tile,dx,dw", GRADIENTS)
def test_gradient_choice(ty, M, K, F, tile, dx, dw):
    notes = made("sdm_ffn_backward", struct(ty, M, K, F), 1)
    assert notes["products"] == [KIND[ty], tile, dx, dw]
    assert notes["grad"][0] == (2 if ty != "f32" and min(M * K, M * F, F * K) <= 4096 else 1)


def test_every_kernel_is_here():
    assert {(ty, t) for ty, *_, t in FORWARDS} == {(ty, t) for ty in ("bf16", "f16", "e4m3") for t in (0, 64, 128, 256)} | {("f32", t) for t in (0, 64, 128)}
    got = {(ty, t, dx > 1, dw > 1) for ty, _, _, _, t, dx, dw in GRADIENTS}
    for ty in ("bf16", "f16", "f32"):
        for t in (64, 128) if ty == "f32" else (64, 128, 256):
            assert (ty, t, False, False) in got and (ty, t, True, False) in got
            assert t == 256 or (ty, t, False, True) in got


def inputs(ty, M, K, F):
    gen = torch.Generator().manual_seed(M + K + F)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    t = TYPES[ty]
    return [v.to(t).cuda() for v in (r(M, K), r(F, K) * K ** -0.5, r(F, K) * K ** -0.5, 0.5 * r(M, F))]


@pytest.mark.gpu
@pytest.mark.parametrize("ty,M,K,F,tile", FORWARDS)
def test_forward(ty, M, K, F, tile):
    say("ffn tiles", ty, M, K, F, tile)
    x, wg, wu, _ = inputs("f32" if ty == "e4m3" else ty, M, K, F)
    s, scales = {}, (None,) * 3
    if ty == "e4m3":
        (x, a), (wg, b), (wu, c) = (sdm.quant_rows(t) for t in (x, wg, wu))
        s, scales = dict(x_scale=a, gate_scale=b, up_scale=c), (a, b, c)
    h, kept = sdm.ffn_forward(x, wg, wu, act="gelu", keep=True, **s)
    want = ffn(x, wg, wu, "gelu", h.dtype, scales)
    for name, v in zip("hgu", (h, *kept)):
        within(v, *want[name], name)


@pytest.mark.gpu
@pytest.mark.parametrize("ty,M,K,F,tile,dx,dw", GRADIENTS)
def test_gradient(ty, M, K, F, tile, dx, dw):
    say("ffn tiles", ty, M, K, F, tile, dx, dw)
    x, wg, wu, dh = inputs(ty, M, K, F)
    kept = sdm.ffn_forward(x, wg, wu, act="silu", keep=True)[1]
    grads = sdm.ffn_backward(dh, x, wg, wu, kept, act="silu")
    want = ffn(x, wg, wu, "silu", x.dtype, dh=dh)
    for name, v in zip(("dx", "dwg", "dwu"), grads):
        within(v, *want[name], name)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [16, 40, 300])
def test_float32_parts_that_leave_out_most(M):
    """1 + 2^-8 - 2^-17 has the parts 1, 2^-8 and -2^-17: the two products left out, of the second and third parts, are 2^-24 of the
    whole together, with one sign. K sums of at most 6 products each round by 2^-24 of what there is."""
    K, F = 256, 50
    v = 1 + 2.0 ** -8 - 2.0 ** -17
    x, w = torch.full((M, K), v, device="cuda"), torch.full((F, K), v, device="cuda")
    g = sdm.ffn_forward(x, w, w, act="none", keep=True)[1][0].double()
    assert ((g - K * v * v).abs() <= (2.0 ** -24 + (6 * K / 16 + 8) * 2.0 ** -24) * K * v * v).all()
