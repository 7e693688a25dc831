"""GPU tests of how far a value that is not finite reaches: what the definition makes of it, and its own chunk of 64 tokens
in its head (and column, for v). Everything else keeps its bits."""

import pytest
import torch

from tests import test_gdr as G

pytestmark = pytest.mark.gpu

AT = 100        # in the second chunk: tokens 64 .. 127


def spread(d, name, bad):
    """Copies of the inputs with one bad value in row 1, head 1 (of its own kind), and what it was put into."""
    e = {n: t.clone() for n, t in d.items()}
    where = (1, AT, 1, 5) if name in "qkv" else (1, AT, 1)
    e[name][where] = bad
    return e


@pytest.mark.parametrize("dk,dv", [(64, 40), (128, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
def test_forward(name, bad, dk, dv):
    print("not finite", name, bad, dk, dv, flush=True)
    d = G.make(3, 200, 2, 4, dk, dv, torch.float32)
    o, s = G.forward(d, 0.125)
    p, t = G.forward(spread(d, name, bad), 0.125)
    hit = torch.zeros_like(o, dtype=torch.bool)
    heads = slice(2, 4) if name in "qk" else slice(1, 2)
    if name == "q":
        hit[1, AT, heads] = True
    else:
        hit[1, 64:, heads] = True
    if name == "v":
        hit[..., :5] = hit[..., 6:] = False
    assert torch.equal(o[~hit], p[~hit])
    after = hit.clone()
    after[:, :AT] = False
    assert not torch.isfinite(p[after]).any()
    state = torch.zeros_like(s, dtype=torch.bool)
    if name != "q":
        state[1, heads] = True
    if name == "v":
        state[..., :5] = state[..., 6:] = False
    assert torch.equal(s[~state], t[~state]) and not torch.isfinite(t[state]).any()


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "do"])
def test_backward_keeps_to_its_sequence_and_key_head(name):
    d = G.make(3, 200, 2, 4, 64, 40, torch.float32)
    a = G.backward(d, 0.125)
    e = {n: t.clone() for n, t in d.items()}
    e[name][(1, AT, 1) + ((5,) if name in ("q", "k", "v", "do") else ())] = float("nan")
    b = G.backward(e, 0.125)
    key = 1 if name in "qk" else 0       # value heads 0 and 1 share key head 0
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x[[0, 2]], y[[0, 2]]), i
        per_key = i < 2
        other = 1 - key if per_key else slice(2, 4) if key == 0 else slice(0, 2)
        if i == 5:
            assert torch.equal(x[1, other], y[1, other]), i
        else:
            assert torch.equal(x[1, :, other], y[1, :, other]), i
    assert not all(torch.isfinite(y[1]).all() for y in b)


def test_tokens_of_no_run_and_idle_states_are_not_read():
    """Packed rows with NaN between and behind the runs; a pool whose unused states are NaN."""
    import deterministic_fp32_gemm_amd as g
    cu = torch.tensor([10, 70, 70, 135], dtype=torch.int32).cuda()
    d = G.make(1, 150, 1, 2, 64, 40, torch.float32, nseq=3)
    e = {n: t.clone() for n, t in d.items()}
    for n in ("q", "k", "v", "g", "beta", "do"):
        e[n][0, :10] = e[n][0, 135:] = float("nan")
    for x, y in zip((*G.forward(d, 0.125, cu_seqlens=cu), *G.backward(d, 0.125, cu_seqlens=cu)),
                    (*G.forward(e, 0.125, cu_seqlens=cu), *G.backward(e, 0.125, cu_seqlens=cu))):
        assert torch.equal(x, y)
    f = G.dev(G.make(3, 1, 2, 4, 64, 40, torch.float32))
    state = torch.full((6, 4, 64, 40), float("nan"), device="cuda")
    state[[4, 1]] = f["s0"][:2]
    slots = torch.tensor([4, -1, 1], dtype=torch.int32).cuda()
    o = g.gdr_step(f["q"], f["k"], f["v"], f["g"], f["beta"], state, slots=slots)
    assert torch.isfinite(o).all() and not o[1].any()
    assert torch.isfinite(state[[4, 1]]).all() and torch.isnan(state[[0, 2, 3, 5]]).all()
