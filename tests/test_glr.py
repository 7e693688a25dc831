"""The gated linear recurrence on the GPU against its definition in 64 bits: types, lengths around its tiles and parts, odd
channels, strides, packed runs, single tokens and the pool of states, values that are not finite, streams and graphs."""

import pytest
import torch

import deterministic_fp32_gemm_amd as sdm
from deterministic_fp32_gemm_amd import block
from tests.block_ref import TYPES, act64, glr, half, within, GATE, U
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def inputs(ty, gty, B, T, D, act, nseq=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n = B if nseq is None else nseq
    g = -torch.nn.functional.softplus(1.5 * r(B, T, D) - 3) - 20.0 * (torch.rand(B, T, D, generator=gen) < 0.02)
    t = dict(x=r(B, T, D).to(TYPES[ty]), g=g.to(TYPES[gty]), z=None if act == "none" else (2 * r(B, T, D)).to(TYPES[ty]),
             h0=r(n, D), dy=r(B, T, D).to(TYPES[ty]), dh=r(n, D))
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def run(t, act, cu=None):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, h, marks = sdm.glr_forward(t["x"], t["g"], t["z"], act=act, initial_state=t["h0"], cu_seqlens=c)
    dx, dg, dz, dh0 = sdm.glr_backward(t["x"], t["g"], t["z"], t["dy"], marks, act=act, initial_state=t["h0"],
                                       dfinal_state=t["dh"], cu_seqlens=c)
    return {"y": y, "state": h, "dx": dx, "dg": dg, "dz": dz, "dh0": dh0}


def check(t, act, cu=None):
    got, want = run(t, act, cu), glr(t["x"], t["g"], t["z"], act, t["h0"], cu, t["dy"], t["dh"])
    for name, (v, bound) in want.items():
        within(got[name], v, bound, name)
    return got


@pytest.mark.parametrize("ty,gty,B,T,D,act", [
    ("f32", "f32", 1, 1, 1, "none"), ("f32", "f32", 3, 15, 5, "silu"), ("bf16", "bf16", 2, 16, 64, "sigmoid"),
    ("f16", "f32", 2, 127, 65, "silu"), ("f32", "f32", 1, 128, 63, "none"), ("bf16", "f32", 1, 129, 130, "silu"),
    ("f16", "f16", 1, 1023, 33, "none"),        # one part less a token, then two parts and more
    ("f32", "f32", 1, 1024, 33, "silu"), ("bf16", "bf16", 1, 1153, 40, "sigmoid"), ("f32", "f32", 1, 3001, 17, "none"),
    ("bf16", "bf16", 2, 1700, 9, "silu"),
])
def test_against_the_definition(ty, gty, B, T, D, act):
    say("glr", ty, gty, B, T, D, act)
    check(inputs(ty, gty, B, T, D, act), act)


@pytest.mark.parametrize("T,cu", [(700, [0, 0, 100, 101, 400, 700]), (5, [0, 5]), (1300, [0, 1299, 1299, 1300]),
                                  (257, [0, 128, 256, 257])])
@pytest.mark.parametrize("ty,act", [("f32", "silu"), ("bf16", "none")])
def test_packed(T, cu, ty, act):
    say("glr packed", T, cu, ty)
    check(inputs(ty, "f32", 1, T, 37, act, len(cu) - 1), act, cu)


@pytest.mark.parametrize("ty,gty,B,T,D,act", [
    ("bf16", "f32", 1, 20001, 70, "silu"),      # tiles from the queue, many groups of them
    ("f16", "f16", 3, 2500, 66, "sigmoid"), ("f32", "f32", 2, 1280, 1, "none"), ("bf16", "bf16", 1, 1024, 4100, "silu"),
])
def test_long_rows(ty, gty, B, T, D, act):
    say("glr long", ty, gty, B, T, D, act)
    check(inputs(ty, gty, B, T, D, act), act)


@pytest.mark.parametrize("ty,act", [("f32", "silu"), ("bf16", "none")])
@pytest.mark.parametrize("lens", [
    [5000] + [30, 0, 1] * 43, [0] * 70 + [3000, 0, 129] + [0] * 70, [128] * 9 + [4096], [100, 4100, 0], [700] * 3])
def test_packed_long_runs(lens, ty, act):
    """Runs taken from the queue and runs walked, with more of them than a wavefront has lanes and empty ones at every place."""
    say("glr packed long", len(lens), sum(lens), ty, act)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    check(inputs(ty, "f32", 1, cu[-1], 65, act, len(lens)), act, cu)


def test_bad_bounds_of_long_runs_stay_inside():
    """As below, where tiles come from the queue: the call ends."""
    t = inputs("f32", "f32", 1, 3000, 12, "silu", 4)
    cu = torch.tensor([-5, 1500, 90, 100000, 7], dtype=torch.int32, device="cuda")
    y, h, marks = sdm.glr_forward(t["x"], t["g"], t["z"], act="silu", initial_state=t["h0"], cu_seqlens=cu)
    sdm.glr_backward(t["x"], t["g"], t["z"], t["dy"], marks, act="silu", initial_state=t["h0"], dfinal_state=t["dh"], cu_seqlens=cu)
    torch.cuda.synchronize()
    assert y.shape == t["x"].shape and marks.shape[1] == 12


def test_two_calls_at_once():
    """Each call has its own queue: two at once on two streams, with strides that are not a tensor's own, give what one gives."""
    base = inputs("bf16", "f32", 2, 6000, 200, "silu")
    t = {k: v.transpose(0, 1).contiguous().transpose(0, 1) if v is not None and v.dim() == 3 else v for k, v in base.items()}
    want = run(base, "silu")
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for s in streams:
            got.append(sdm.glr_forward(t["x"], t["g"], t["z"], act="silu", initial_state=t["h0"], stream=s)[:2])
    torch.cuda.synchronize()
    for y, h in got:
        assert torch.equal(y, want["y"]) and torch.equal(h, want["state"])


def test_the_same_bits_from_the_queue():
    t, cu = inputs("bf16", "f32", 1, 9000, 300, "silu", 3), [0, 8000, 8100, 9000]
    want = run(t, "silu", cu)
    for _ in range(5):
        got = run(t, "silu", cu)
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_tokens_of_no_run_are_zero():
    t = inputs("f32", "f32", 1, 300, 20, "silu", 2)
    got = run(t, "silu", [10, 150, 290])
    part = {k: (v[:, 10:290].contiguous() if v is not None and v.dim() == 3 else v) for k, v in t.items()}
    want = run(part, "silu", [0, 140, 280])
    for name in ("y", "dx", "dg", "dz"):
        assert torch.equal(got[name][:, 10:290], want[name])
        assert not got[name][:, :10].any() and not got[name][:, 290:].any()
    assert torch.equal(got["state"], want["state"]) and torch.equal(got["dh0"], want["dh0"])


def test_without_states():
    t = inputs("f32", "f32", 2, 40, 10, "none")
    t["h0"] = t["dh"] = None
    check(t, "none")


def test_empty():
    x = torch.zeros(2, 0, 8, device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    y, h, marks = sdm.glr_forward(x, x, initial_state=h0)
    assert y.shape == x.shape and torch.equal(h, h0) and marks.shape == (0, 8)
    dx, dg, dz, dh0 = sdm.glr_backward(x, x, None, x, marks, initial_state=h0, dfinal_state=2 * h0)
    assert dx.shape == x.shape and dz is None and torch.equal(dh0, 2 * h0)
    t = inputs("f32", "f32", 1, 3, 8, "none", 2)
    got = run(t, "none", [0, 0, 0])
    assert torch.equal(got["state"], t["h0"]) and torch.equal(got["dh0"], t["dh"]) and not got["y"].any()


def test_strides_and_alignment():
    """The parts of one projection, a batch that lies token by token, and a last axis that is not contiguous."""
    t = inputs("bf16", "bf16", 2, 200, 30, "silu")
    want = run(t, "silu")
    whole = torch.zeros(200, 2, 91, dtype=torch.bfloat16, device="cuda")
    v = dict(t)
    for i, k in enumerate(("x", "g", "z")):
        view = whole[:, :, 1 + 30 * i:31 + 30 * i].transpose(0, 1)
        view.copy_(t[k])
        v[k] = view
    v["dy"] = torch.empty(2, 30, 200, dtype=torch.bfloat16, device="cuda").transpose(1, 2).copy_(t["dy"])
    got = run(v, "silu")
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_the_same_bits_again():
    t = inputs("bf16", "f32", 1, 5000, 70, "silu")
    a, b = run(t, "silu"), run(t, "silu")
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("where", [0, 130, 1500])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_not_finite_stays_in_its_channel(where, value):
    """A value that is not finite reaches the later tokens of its channel and run (earlier ones in the gradient), no others."""
    t = inputs("f32", "f32", 1, 1600, 6, "silu", 2)
    cu = [0, 1550, 1600]
    want = run(t, "silu", cu)
    t["x"][0, where, 2] = value
    got = run(t, "silu", cu)
    other = [0, 1, 3, 4, 5]
    for k in ("y", "dx", "dg", "dz"):
        assert torch.equal(got[k][..., other], want[k][..., other])
        assert torch.equal(got[k][:, 1550:], want[k][:, 1550:])
    assert torch.equal(got["y"][:, :where], want["y"][:, :where]) and torch.equal(got["dx"], want["dx"])
    assert not torch.isfinite(got["y"][0, where, 2])


def test_forgetting_and_growing():
    t = inputs("f32", "f32", 1, 1300, 4, "none")
    t["g"][0, 700] = -float("inf")
    got = run(t, "none")
    assert torch.isfinite(got["y"]).all() and torch.equal(got["y"][0, 700], t["x"][0, 700])
    assert not got["dg"][0, 700].any()
    # from an empty state a growth beyond float32 makes nothing
    x, g = torch.zeros(1, 1300, 4, device="cuda"), torch.full((1, 1300, 4), 3.0, device="cuda")
    assert not sdm.glr_forward(x, g)[0].any()


@pytest.mark.parametrize("ty,gty,B,T,D,act,pool", [("f32", "f32", 1, 1, 1, "none", 1), ("bf16", "f32", 5, 1, 257, "silu", 9),
                                                   ("f16", "f16", 3, 4, 100, "sigmoid", 3), ("bf16", "bf16", 70, 2, 513, "none", 90)])
def test_step(ty, gty, B, T, D, act, pool):
    say("glr step", ty, gty, B, T, D, act, pool)
    t = inputs(ty, gty, B, T, D, act)
    state = torch.randn(pool, D, device="cuda")
    slots = torch.randperm(pool)[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, pool
    before, live = state.clone(), [b for b in range(B) if 0 <= slots[b] < pool]
    y = sdm.glr_step(t["x"], t["g"], t["z"], state, act=act, slots=slots.cuda())
    want = glr(t["x"], t["g"], t["z"], act, before[slots.long().clamp(0, pool - 1).cuda()])
    within(y[live], want["y"][0][live], want["y"][1][live], "y")
    within(state[slots[live].long().cuda()], want["state"][0][live], want["state"][1][live], "state")
    idle = [b for b in range(B) if b not in live]
    assert not y[idle].any()
    rest = torch.ones(pool, dtype=torch.bool)
    rest[slots[live].long()] = False
    assert torch.equal(state[rest.cuda()], before[rest.cuda()])


def test_steps_follow_the_sequence():
    """A prompt, then token by token: the states of the whole sequence."""
    t = inputs("f32", "f32", 2, 140, 70, "silu")
    want = glr(t["x"], t["g"], t["z"], "silu", t["h0"])
    y, state, _ = sdm.glr_forward(t["x"][:, :130], t["g"][:, :130], t["z"][:, :130], act="silu", initial_state=t["h0"])
    ys = [y] + [sdm.glr_step(*(t[k][:, i:i + 1] for k in ("x", "g", "z")), state, act="silu") for i in range(130, 140)]
    within(torch.cat(ys, 1), *want["y"], "y")
    within(state, *want["state"], "state")


def test_rows_around_are_left_alone():
    """The C entry's strided outputs: what lies between and behind the rows keeps its bits."""
    import ctypes
    t = inputs("f32", "f32", 1, 150, 20, "none")
    whole = torch.full((152, 32), 7.0, device="cuda")
    y = whole[1:151, 5:25]
    want, h, _ = sdm.glr_forward(t["x"], t["g"], initial_state=t["h0"])
    a = block.sdm_glr_args_t(dtype=0, gtype=0, act=0, B=1, T=150, D=20, nseq=1)
    a.x, a.g = block.sdm_seq_t(t["x"].data_ptr(), 3000, 20), block.sdm_seq_t(t["g"].data_ptr(), 3000, 20)
    a.y, a.h0 = block.sdm_seq_t(y.data_ptr(), 150 * 32, 32), t["h0"].data_ptr()
    assert block.load().sdm_glr_forward(ctypes.byref(a), None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y, want[0])
    y.fill_(7.0)
    assert (whole == 7.0).all()


def test_bad_bounds_stay_inside():
    """Bounds out of range and out of order are clamped: nothing outside the buffers is touched."""
    t = inputs("f32", "f32", 1, 200, 12, "silu", 4)
    cu = torch.tensor([-5, 150, 90, 1000, 7], dtype=torch.int32, device="cuda")
    guard = torch.full((4096,), 3.0, device="cuda")
    y, h, marks = sdm.glr_forward(t["x"], t["g"], t["z"], act="silu", initial_state=t["h0"], cu_seqlens=cu)
    sdm.glr_backward(t["x"], t["g"], t["z"], t["dy"], marks, act="silu", initial_state=t["h0"], dfinal_state=t["dh"], cu_seqlens=cu)
    torch.cuda.synchronize()
    assert (guard == 3.0).all()
    want = sdm.glr_forward(t["x"][:, :150], t["g"][:, :150], t["z"][:, :150], act="silu", initial_state=t["h0"][:1])
    assert torch.equal(h[0], want[1][0])


def test_streams_and_graphs():
    t = inputs("bf16", "f32", 1, 2100, 70, "silu")
    want = run(t, "silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, marks = sdm.glr_forward(t["x"], t["g"], t["z"], act="silu", initial_state=t["h0"], stream=side)
    grads = sdm.glr_backward(t["x"], t["g"], t["z"], t["dy"], marks, act="silu", initial_state=t["h0"], dfinal_state=t["dh"], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want["y"]) and all(torch.equal(a, want[k]) for a, k in zip(grads, ("dx", "dg", "dz", "dh0")))
    graph = torch.cuda.CUDAGraph()
    run(t, "silu")
    with torch.cuda.graph(graph):
        got = run(t, "silu")
    for i in range(3):
        fresh = inputs("bf16", "f32", 1, 2100, 70, "silu", seed=i + 1)
        for k in t:
            t[k].copy_(fresh[k])
        graph.replay()
        torch.cuda.synchronize()
        want = run(fresh, "silu")
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_gradients_through_the_graph_and_differences():
    t = inputs("f32", "f32", 1, 20, 3, "silu")
    leaves = {k: t[k].clone().requires_grad_() for k in ("x", "g", "z", "h0")}
    y, h, marks = sdm.glr_forward(leaves["x"], leaves["g"], leaves["z"], act="silu", initial_state=leaves["h0"])
    assert not marks.requires_grad
    torch.autograd.backward([y, h], [t["dy"], t["dh"]])
    want = run(t, "silu")
    for k, n in (("x", "dx"), ("g", "dg"), ("z", "dz"), ("h0", "dh0")):
        assert torch.equal(leaves[k].grad, want[n])
    # differences of the definition itself, in 64 bits, along each leaf's own direction
    for k, n in (("x", "dx"), ("g", "dg"), ("z", "dz"), ("h0", "dh0")):
        gen = torch.Generator().manual_seed(1)
        d = torch.randn(t[k].shape, generator=gen).double()
        def loss(s):
            u = {m: t[m].double().cpu() for m in ("x", "g", "z", "h0")}
            u[k] = u[k] + s * d
            c, total = u["h0"][0], 0.0
            for i in range(20):
                c = u["g"][0, i].exp() * c + u["x"][0, i]
                total = total + (t["dy"][0, i].double().cpu() * c * act64(u["z"][0, i], "silu")[0]).sum()
            return total + (t["dh"][0].double().cpu() * c).sum()
        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = (want[n].double().cpu() * d).sum()
        # a gradient's own bound is some 2^-20 of its largest terms; the difference's error is 1e-10 of third derivatives
        assert abs(slope - got) <= 1e-5 * (want[n].double().cpu().abs() * d.abs()).sum()


def test_another_device_or_type_is_refused():
    t = inputs("f32", "f32", 1, 5, 4, "none")
    with pytest.raises(ValueError):
        sdm.glr_forward(t["x"], t["g"].cpu())
    with pytest.raises(TypeError):
        sdm.glr_forward(t["x"], t["g"].bfloat16())
    y, h, marks = sdm.glr_forward(t["x"], t["g"])
    with pytest.raises(ValueError):
        sdm.glr_backward(t["x"], t["g"], None, t["dy"], marks[:0])
