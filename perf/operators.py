"""The gated delta rule and the block norm: what is measured, their plain forms and their definitions in 64 bits.

The gated delta rule (one state S of dk x dv per sequence and value head, r = Hv / Hk value heads sharing a q/k head):

    S' = exp(g_t) S_{t-1};  u_t = beta_t (v_t - S'^T k_t);  S_t = S' + k_t u_t^T;  o_t = scale S_t^T q_t

in three forms: over whole sequences (gdr_forward), its gradient (gdr_backward), and one or a few tokens against a pool
of states updated in place (gdr_step). The block norm closes a residual block and opens the next:

    n = o rsqrt(mean o^2 + eps) w_post;  x' = x + s n act(z);  y = x' rsqrt(mean x'^2 + eps) w_pre

forward (norm_forward) and backward (norm_backward).
"""
import math
import random

import torch

own = False

C = 64              # tokens a chunk of the plain chunked form: the chunk length of this library's workloads
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a few short sequences in float32: latency of the chunked form
        {"name": "fwd_short_f32", "op": "fwd", "type": "f32", "B": 2, "T": 100, "Hk": 2, "Hv": 4, "dk": 64, "dv": 64, "nseq": 0},
        # a long prompt, 32 value heads over 16 shared key heads: prefill
        {"name": "fwd_long_bf16", "op": "fwd", "type": "bf16", "B": 1, "T": 16384, "Hk": 16, "Hv": 32, "dk": 128, "dv": 128, "nseq": 0},
        # packed sequences of odd lengths, head sizes off the tile sizes
        {"name": "fwd_ragged_f16", "op": "fwd", "type": "f16", "B": 1, "T": 9001, "Hk": 8, "Hv": 8, "dk": 72, "dv": 100, "nseq": 23},
        # gradients of an odd length with odd head sizes
        {"name": "bwd_odd_f32", "op": "bwd", "type": "f32", "B": 1, "T": 333, "Hk": 3, "Hv": 3, "dk": 40, "dv": 56, "nseq": 0},
        # a training step's layer: two sequences, shared key heads
        {"name": "bwd_train_bf16", "op": "bwd", "type": "bf16", "B": 2, "T": 4096, "Hk": 8, "Hv": 16, "dk": 128, "dv": 128, "nseq": 0},
        # float32 training with wide value heads (64 x 256, the largest workload's chunk shape)
        {"name": "bwd_wide_f32", "op": "bwd", "type": "f32", "B": 4, "T": 1024, "Hk": 4, "Hv": 4, "dk": 64, "dv": 256, "nseq": 0},
        # one stream's next token: latency
        {"name": "step_one_bf16", "op": "step", "type": "bf16", "B": 1, "T": 1, "Hk": 8, "Hv": 16, "dk": 128, "dv": 128, "pool": 4},
        # a full serving batch's next token, slots scattered over the pool, some streams idle
        {"name": "step_batch_bf16", "op": "step", "type": "bf16", "B": 256, "T": 1, "Hk": 16, "Hv": 32, "dk": 128, "dv": 128, "pool": 320},
        # the norm of a decode batch: latency
        {"name": "norm_decode_bf16", "op": "norm", "type": "bf16", "rows": 16, "D": 2048, "act": "silu"},
        # the norm of a training batch
        {"name": "norm_train_bf16", "op": "norm", "type": "bf16", "rows": 16384, "D": 4096, "act": "silu"},
        # gradients of an odd row length in float32
        {"name": "norm_bwd_odd_f32", "op": "norm_bwd", "type": "f32", "rows": 777, "D": 1111, "act": "sigmoid"},
        # gradients of a training batch
        {"name": "norm_bwd_train_bf16", "op": "norm_bwd", "type": "bf16", "rows": 16384, "D": 4096, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "norm_bwd"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("norm", "norm_bwd"):
        D = _log(rng, 48, 8192)
        rows = min(_log(rng, 1, 16384), 16384 * 4096 // D)
        return {"op": op, "type": kind, "rows": rows, "D": D, "act": rng.choice(["none", "sigmoid", "silu"])}
    dk, dv = (rng.choice([32, 64, 96, 128, rng.randint(17, 160)]) for _ in range(2))
    Hk, r = rng.randint(1, 8), rng.choice([1, 1, 2, 3])
    if op == "step":
        B = _log(rng, 1, 200)
        return {"op": op, "type": kind, "B": B, "T": rng.choice([1, 1, 1, 2, 3]), "Hk": Hk, "Hv": Hk * r, "dk": dk, "dv": dv, "pool": B + rng.randint(0, 40)}
    T = _log(rng, 1, 16384 if op == "fwd" else 4096)
    nseq = rng.choice([0, 0, rng.randint(1, 24)])
    B = 1 if nseq else max(1, min(rng.randint(1, 4), 16384 // T))
    return {"op": op, "type": kind, "B": B, "T": T, "Hk": Hk, "Hv": Hk * r, "dk": dk, "dv": dv, "nseq": nseq}


def _lengths(case):
    """The lengths of a packed case's sequences: odd ones, short ones and now and then an empty one."""
    rng = random.Random("%d %d" % (case["T"], case["nseq"]))
    cuts = sorted(rng.randint(0, case["T"]) for _ in range(case["nseq"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    ty = TYPES[case["type"]]

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        s |= {k: rnd(R, D).to(ty) for k in ("x", "o", "z")}
        if case["act"] == "none":
            s["z"] = None
        s |= {"w_post": (1 + 0.2 * rnd(D)).to(ty), "w_pre": (1 + 0.2 * rnd(D)).to(ty), "scale": (0.5 + 0.1 * rnd(D)).to(ty)}
        if case["op"] == "norm_bwd":
            # what the forward call left: the new residual and each row's two reciprocal norms
            s["xn"], _, s["rstd"] = _norm_plain(s)
            s |= {"dy": (0.01 * rnd(R, D)).to(ty), "dxn": (0.01 * rnd(R, D)).to(ty)}
        return s
    B, T, Hk, Hv, dk, dv = (case[k] for k in ("B", "T", "Hk", "Hv", "dk", "dv"))
    q, k = rnd(B, T, Hk, dk), rnd(B, T, Hk, dk)
    s["q"] = (q / q.norm(dim=-1, keepdim=True)).to(ty)      # q and k come normalised, as such layers have them
    s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(ty)
    s["v"] = rnd(B, T, Hv, dv).to(ty)
    # log decays from gentle to strong, and one token in 50 that all but forgets
    s["g"] = -torch.nn.functional.softplus(rnd(B, T, Hv) * 1.5 - 3)
    s["g"] -= 20.0 * (torch.rand(B, T, Hv, generator=gen, device="cuda") < 0.02)
    s["beta"] = torch.sigmoid(rnd(B, T, Hv))
    s["sm"] = dk ** -0.5
    if case["op"] == "step":
        s["state"] = 0.1 * rnd(case["pool"], Hv, dk, dv)
        slots = torch.randperm(case["pool"], generator=gen, device="cuda")[:B].to(torch.int32)
        if B > 8:
            slots[torch.randint(B, (B // 16,), generator=gen, device="cuda")] = -1      # idle streams
        s["slots"] = slots
        return s
    n = case["nseq"] or B
    s["cu"], s["longest"] = None, T
    if case["nseq"]:
        lens = _lengths(case)
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["longest"] = max(lens)
    s["s0"] = 0.1 * rnd(n, Hv, dk, dv)
    if case["op"] == "bwd":
        s["do"] = (0.1 * rnd(B, T, Hv, dv)).to(ty)
        s["ds"] = 0.02 * rnd(n, Hv, dk, dv)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import deterministic_fp32_gemm_amd as g
        if op == "fwd":
            return g.gdr_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["sm"], initial_state=s["s0"], cu_seqlens=s["cu"])
        if op == "bwd":
            return g.gdr_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], scale=s["sm"], initial_state=s["s0"], dfinal_state=s["ds"], cu_seqlens=s["cu"])
        if op == "step":
            return g.gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], scale=s["sm"]), s["state"]
        if op == "norm":
            return g.norm_forward(s["x"], s["o"], s["z"], s["w_post"], s["w_pre"], s["scale"], act=s["case"]["act"], eps=EPS)
        return g.norm_backward(s["dxn"], s["dy"], s["xn"], s["o"], s["z"], s["w_post"], s["w_pre"], s["scale"], s["rstd"], act=s["case"]["act"])
    return {"fwd": _fwd_plain, "bwd": _bwd_plain, "step": _step_plain, "norm": _norm_plain, "norm_bwd": _norm_bwd_plain}[op](s)


# ---- plain forms: 32 bits, elementary operations --------------------------------------------------------------------
def _rows(s):
    """(index of each padded place among the tokens, whether it holds a token), for sequences padded to whole chunks."""
    B, T = s["q"].shape[:2]
    n, pad = s["s0"].shape[0], -(-s["longest"] // C) * C
    at = torch.arange(pad, device="cuda")[None]
    if s["cu"] is None:
        start, length = torch.arange(B, device="cuda")[:, None] * T, torch.full((B, 1), T, device="cuda")
    else:
        start, length = s["cu"][:-1, None].long(), (s["cu"][1:] - s["cu"][:-1])[:, None].long()
    held = (at < length) & (start + at < B * T)
    return torch.where(held, start + at, 0), held, n, pad


def _chunked(x, rows, held, heads):
    """[B, T, h, d] or [B, T, h] tokens -> float32 [n, heads, chunks, C, d], shared heads repeated, zeros where there is no token."""
    x = x.flatten(0, 1)[rows].float()
    x = x * held.reshape(held.shape + (1,) * (x.dim() - 2))
    x = x.repeat_interleave(heads // x.shape[2], dim=2)
    x = x if x.dim() == 4 else x[..., None]
    return x.transpose(1, 2).unflatten(2, (-1, C)).contiguous()


def _flat(x, held, like):
    """Back from chunks to the tokens of `like`'s shape and type, shared heads summed."""
    n, H, N, _, d = x.shape
    x = x.flatten(2, 3).transpose(1, 2)[held]
    h = like.shape[2]
    x = x.unflatten(1, (h, H // h)).sum(2)
    return x.reshape(like.shape).to(like.dtype)


def _intra(s):
    """What a chunk's tokens alone determine, for all chunks at once."""
    rows, held, n, pad = _rows(s)
    Hv = s["v"].shape[2]
    q, k, v, g, beta = (_chunked(s[x], rows, held, Hv) for x in ("q", "k", "v", "g", "beta"))
    G = g.double().cumsum(3)
    low = torch.tril(torch.ones(C, C, dtype=torch.bool, device="cuda"))
    decay = torch.where(low, G - G.transpose(3, 4), -math.inf).exp().float()
    kk = k @ k.transpose(3, 4)
    A = beta * kk * decay * (1 - torch.eye(C, device="cuda"))
    inv = torch.eye(C, device="cuda").expand_as(A).contiguous()
    for i in range(1, C):
        inv[..., i, :] -= (A[..., i, None, :i] @ inv[..., :i, :])[..., 0, :]
    return dict(q=q, k=k, v=v, beta=beta, held=held, decay=decay, kk=kk, inv=inv, eG=G.exp().float(), last=(G[..., -1:, :] - G).exp().float(),
                whole=G[..., -1, :].exp().float()[..., None], P=s["sm"] * decay * (q @ k.transpose(3, 4)))


def _states(s, c):
    """Each chunk's entering state, its u, and the state after the last."""
    S, kept, us = s["s0"].clone(), [], []
    for j in range(c["q"].shape[2]):
        kept.append(S)
        r = c["beta"][:, :, j] * (c["v"][:, :, j] - c["eG"][:, :, j] * (c["k"][:, :, j] @ S))
        u = c["inv"][:, :, j] @ r
        S = c["whole"][:, :, j] * S + (c["last"][:, :, j] * c["k"][:, :, j]).transpose(2, 3) @ u
        us.append(u)
    return torch.stack(kept, 2), torch.stack(us, 2), S


def _fwd_plain(s):
    if not s["longest"]:
        return torch.zeros_like(s["v"]), s["s0"].clone()
    c = _intra(s)
    S, u, final = _states(s, c)
    o = s["sm"] * c["eG"] * (c["q"] @ S) + c["P"] @ u
    return _flat(o, c["held"], s["v"]), final


def _bwd_plain(s):
    c = _intra(s)
    S, u, _ = _states(s, c)
    q, k, v, beta, eG, last, P = (c[x] for x in ("q", "k", "v", "beta", "eG", "last", "P"))
    do = _chunked(s["do"], *_rows(s)[:2], v.shape[1])
    dS, kept, dR = s["ds"].clone(), [], []
    du0, tr = P.transpose(3, 4) @ do, c["inv"].transpose(3, 4)
    qdo = s["sm"] * (eG * q).transpose(3, 4) @ do
    for j in reversed(range(q.shape[2])):
        kept.append(dS)
        r = tr[:, :, j] @ (du0[:, :, j] + last[:, :, j] * (k[:, :, j] @ dS))
        dS = c["whole"][:, :, j] * dS + qdo[:, :, j] - (beta * eG * k)[:, :, j].transpose(2, 3) @ r
        dR.append(r)
    dE, dR = torch.stack(kept[::-1], 2), torch.stack(dR[::-1], 2)     # gradients of each chunk's last state and of r
    dP = do @ u.transpose(3, 4) * c["decay"]
    dA = -(dR @ u.transpose(3, 4)) * c["decay"] * (1 - torch.eye(C, device="cuda"))
    dq = s["sm"] * (eG * (do @ S.transpose(3, 4)) + dP @ k)
    dkr = dA @ k - eG * (dR @ S.transpose(3, 4))                      # beta times this is k's own row's part
    dks = last * (u @ dE.transpose(3, 4))
    dkc = s["sm"] * dP.transpose(3, 4) @ q + dks
    dkb = (dA * beta).transpose(3, 4) @ k
    dbeta = (dR * v).sum(-1, keepdim=True) + (k * dkr).sum(-1, keepdim=True)
    dG = (q * dq + k * (beta * dkr - dkc - dkb)).double().sum(-1, keepdim=True)
    dG[..., -1, :] += (k * dks).double().sum((3, 4))[..., None] + (c["whole"] * (S * dE)).double().sum((3, 4))[..., None]
    dg = dG.flip(3).cumsum(3).flip(3)
    dk = beta * dkr + dkc + dkb
    held = c["held"]
    return (_flat(dq, held, s["q"]), _flat(dk, held, s["k"]), _flat(beta * dR, held, s["v"]), _flat(dg, held, s["g"]), _flat(dbeta, held, s["beta"]), dS)


def _step_plain(s):
    Hv = s["v"].shape[2]
    live = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    S = s["state"][at]
    q, k = (s[x].float().repeat_interleave(Hv // s[x].shape[2], dim=2) for x in ("q", "k"))
    out = []
    for t in range(q.shape[1]):
        S = S * s["g"][:, t].exp()[..., None, None]
        kt = k[:, t, :, :, None]
        u = s["beta"][:, t, :, None] * (s["v"][:, t].float() - (S * kt).sum(2))
        S = S + kt * u[:, :, None]
        out.append(s["sm"] * (S * q[:, t, :, :, None]).sum(2))
    o = torch.stack(out, 1) * live[:, None, None, None]
    s["state"][at[live]] = S[live]
    return o.to(s["v"].dtype), s["state"]


def _gate(z, act):
    if act == "none":
        return 1.0, None
    z = z.float()
    p = 1 / (1 + torch.exp(-z))
    return (p, p * (1 - p)) if act == "sigmoid" else (z * p, p * (1 + z * (1 - p)))


def _norm_plain(s):
    x, o, w1, w2, sc = (s[k].float() for k in ("x", "o", "w_post", "w_pre", "scale"))
    r1 = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)
    xn = (x + sc * (o * r1 * w1 * _gate(s["z"], s["case"]["act"])[0])).to(s["x"].dtype)
    # y is the norm of the residual as it is stored: what the next block reads
    r2 = torch.rsqrt((xn.float() * xn.float()).mean(-1, keepdim=True) + EPS)
    return xn, (xn.float() * r2 * w2).to(xn.dtype), torch.cat([r1, r2], 1)


def _norm_bwd_plain(s):
    xn, o, w1, w2, sc, dy, dxn = (s[k].float() for k in ("xn", "o", "w_post", "w_pre", "scale", "dy", "dxn"))
    r1, r2 = s["rstd"][:, :1], s["rstd"][:, 1:]
    t = dy * w2
    dx = dxn + r2 * (t - xn * r2 * r2 * (t * xn).mean(-1, keepdim=True))
    a, da = _gate(s["z"], s["case"]["act"])
    n = o * r1
    dn = dx * sc * a
    t = dn * w1
    do = r1 * (t - n * (t * n).mean(-1, keepdim=True))
    ty, wt = s["x"].dtype, s["w_pre"].dtype
    return (dx.to(ty), do.to(ty), None if da is None else (dx * sc * n * w1 * da).to(ty), (dn * n).sum(0).to(wt), (dy * xn * r2).sum(0).to(wt), (dx * n * w1 * a).sum(0).to(wt))


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "step":
        return _exact_step(s)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_bwd":
        return _exact_norm_bwd(s)
    return _exact_gdr(s, case["op"] == "bwd")


def _exact_gdr(s, backward):
    """The recurrence token by token, all sequences side by side; a sequence that has ended stands still."""
    B, T, Hv, dv = s["v"].shape
    dk, n, L = s["q"].shape[3], s["s0"].shape[0], s["longest"]
    if s["cu"] is None:
        first, many = [b * T for b in range(B)], [T] * B
    else:
        c = s["cu"].tolist()
        first, many = c[:-1], [b - a for a, b in zip(c, c[1:])]
    src = torch.zeros(n, L, dtype=torch.long, device="cuda")
    on = torch.zeros(n, L, dtype=torch.float64, device="cuda")
    for i in range(n):
        src[i, : many[i]] = torch.arange(first[i], first[i] + many[i], device="cuda")
        on[i, : many[i]] = 1

    def lay(x):
        x = x.reshape(B * T, *x.shape[2:]).double()[src]
        x = x.repeat_interleave(Hv // x.shape[2], 2)
        return (x * (on[..., None] if x.dim() == 3 else on[..., None, None])).transpose(0, 1).contiguous()      # [L, n, Hv, ...]

    q, k, v, g, beta = (lay(s[x]) for x in ("q", "k", "v", "g", "beta"))
    a = g.exp()
    if backward and L * n * Hv * dk * dv * 8 > 60e9:
        return None
    S, o, past = s["s0"].double(), [], []
    for t in range(L):
        S = S * a[t][..., None, None]
        if backward:
            past.append(S)
        u = beta[t][..., None] * (v[t] - torch.matmul(k[t][..., None, :], S)[..., 0, :])
        S = S + k[t][..., None] * u[..., None, :]
        if not backward:
            o.append(torch.matmul(q[t][..., None, :], S)[..., 0, :])

    def back(x, like):
        x = x.transpose(0, 1)
        x = x.unflatten(2, (like.shape[2], -1)).sum(3) if x.shape[2] != like.shape[2] else x
        out = torch.zeros(B * T, *x.shape[2:], dtype=torch.float64, device="cuda")
        out[src[on > 0]] = x[on > 0]
        return out.reshape(like.shape)

    if not backward:
        return (back(s["sm"] * torch.stack(o), s["v"]) if L else s["v"].double()), S
    do = lay(s["do"]) * s["sm"]
    D = s["ds"].double()
    dq, dk_, dv_, dg, db = [], [], [], [], []
    for t in reversed(range(L)):
        Sp = past.pop()
        e = v[t] - torch.matmul(k[t][..., None, :], Sp)[..., 0, :]
        u = beta[t][..., None] * e
        after = Sp + k[t][..., None] * u[..., None, :]
        dq.append(torch.matmul(after, do[t][..., None])[..., 0])
        D = D + q[t][..., None] * do[t][..., None, :]
        du = torch.matmul(k[t][..., None, :], D)[..., 0, :]
        db.append((du * e).sum(-1))
        dr = beta[t][..., None] * du
        dv_.append(dr)
        dk_.append(torch.matmul(D, u[..., None])[..., 0] - torch.matmul(Sp, dr[..., None])[..., 0])
        D = D - k[t][..., None] * dr[..., None, :]
        dg.append((D * Sp).sum((-1, -2)))
        D = D * a[t][..., None, None]
    turn = lambda x, like: back(torch.stack(x[::-1]), like)  # noqa: E731
    return turn(dq, s["q"]), turn(dk_, s["k"]), turn(dv_, s["v"]), turn(dg, s["g"]), turn(db, s["beta"]), D


def _exact_step(s):
    Hv = s["v"].shape[2]
    r = Hv // s["q"].shape[2]
    state = s["state"].double()
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    use = torch.nonzero(s["slots"] >= 0)[:, 0]
    S = state[s["slots"][use].long()]
    for t in range(s["q"].shape[1]):
        q, k = (s[x][use, t].double().repeat_interleave(r, 1) for x in ("q", "k"))
        S = S * torch.exp(s["g"][use, t].double())[:, :, None, None]
        e = s["v"][use, t].double() - torch.matmul(k[:, :, None, :], S)[:, :, 0]
        S = S + k[..., None] * (s["beta"][use, t].double()[..., None] * e)[:, :, None, :]
        o[use, t] = s["sm"] * torch.matmul(q[:, :, None, :], S)[:, :, 0]
    state[s["slots"][use].long()] = S
    return o, state


def _act64(z, act):
    return 1.0 if act == "none" else torch.sigmoid(z) * (z if act == "silu" else 1)


def _exact_norm(s):
    x, o, w1, w2, sc = (s[k].double() for k in ("x", "o", "w_post", "w_pre", "scale"))
    z = None if s["z"] is None else s["z"].double()
    m1 = (o.square().mean(-1, keepdim=True) + EPS).sqrt()
    xn = x + sc * w1 * o / m1 * _act64(z, s["case"]["act"])
    kept = xn.to(s["x"].dtype).double()
    m2 = (kept.square().mean(-1, keepdim=True) + EPS).sqrt()
    return xn, kept / m2 * w2, torch.cat([1 / m1, 1 / m2], 1)


def _exact_norm_bwd(s):
    """Differentiated by machine from the definition, at the residual that the forward call stored."""
    o, w1, w2, sc, xn = (s[k].double().requires_grad_() for k in ("o", "w_post", "w_pre", "scale", "xn"))
    z = None if s["z"] is None else s["z"].double().requires_grad_()
    y = xn / (xn.square().mean(-1, keepdim=True) + EPS).sqrt() * w2
    dx, dw2 = torch.autograd.grad(y, (xn, w2), s["dy"].double())
    dx = dx + s["dxn"].double()
    add = sc * w1 * o / (o.square().mean(-1, keepdim=True) + EPS).sqrt() * _act64(z, s["case"]["act"])
    do, dw1, dsc, *dz = torch.autograd.grad(add, (o, w1, sc) + (() if z is None else (z,)), dx)
    dz = dz[0] if dz else None
    return dx, do, dz, dw1, dw2, dsc


def work(case):
    t = {"f32": 4, "bf16": 2, "f16": 2}[case["type"]]
    if case["op"] in ("norm", "norm_bwd"):
        n = case["rows"] * case["D"]
        back, gate = case["op"] == "norm_bwd", case["act"] != "none"
        return {"bytes": ((6 + 2 * gate) if back else 4 + gate) * n * t + (6 if back else 3) * case["D"] * t + 8 * case["rows"], "flops": (30 if back else 14) * n}
    B, T, Hk, Hv, dk, dv = (case[k] for k in ("B", "T", "Hk", "Hv", "dk", "dv"))
    n, state = B * T, Hv * dk * dv
    token = (2 * Hk * dk + Hv * dv) * t + 8 * Hv            # q, k, v, g and beta of one token
    if case["op"] == "step":
        live = B - (B // 16 if B > 8 else 0)
        return {"bytes": n * (token + Hv * dv * t) + 8 * live * state, "flops": 7 * n * state}
    seqs = case["nseq"] or B
    if case["op"] == "fwd":
        return {"bytes": n * (token + Hv * dv * t) + 8 * seqs * state, "flops": 6 * n * state}
    return {"bytes": n * (2 * token + Hv * dv * t) + 12 * seqs * state, "flops": 18 * n * state}
