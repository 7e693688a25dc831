"""The gated linear recurrence, the norm with an 8-bit output and the gated feed-forward product: what is measured, their
plain forms and their definitions in 64 bits.

The gated linear recurrence (one float32 state a channel) over whole sequences, as a training step (forward and
gradient), and one or a few tokens against a pool of states updated in place:

    h_t = exp(g_t) h_{t-1} + x_t;  y_t = h_t act(z_t)

The norm with the residual's addition and an output in 8 bits, and the same rounding alone for weights:

    x' = x + r;  y = x' rsqrt(mean x'^2 + eps) w;  s = max(max |y| / 448, 2^-126);  q = e4m3(y / s)

The gated feed-forward product, forward and as a training step (forward and gradient):

    h = act(x Wg^T) * (x Wu^T)
"""
import math
import random

import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # a long prompt through one layer, gated output: prefill
        {"name": "rec_prompt_bf16", "op": "rec", "type": "bf16", "gtype": "f32", "B": 1, "T": 16384, "D": 4096, "act": "silu", "nseq": 0},
        # packed sequences of odd lengths in float32, an odd number of channels, no output gate
        {"name": "rec_ragged_f32", "op": "rec", "type": "f32", "gtype": "f32", "B": 1, "T": 9001, "D": 1001, "act": "none", "nseq": 23},
        # a training step's layer: four sequences, forward and gradient
        {"name": "rec_train_bf16", "op": "rec_train", "type": "bf16", "gtype": "bf16", "B": 4, "T": 4096, "D": 4096, "act": "silu", "nseq": 0},
        # a full serving batch's next token, slots scattered over the pool, some streams idle
        {"name": "rec_step_bf16", "op": "rec_step", "type": "bf16", "gtype": "f32", "B": 256, "T": 1, "D": 4096, "act": "silu", "pool": 320},
        # the norm before a feed-forward of a decode batch: latency
        {"name": "quant_decode_bf16", "op": "quant", "type": "bf16", "rows": 16, "D": 2048, "res": True},
        # the norm of a prefill
        {"name": "quant_prefill_bf16", "op": "quant", "type": "bf16", "rows": 16384, "D": 4096, "res": True},
        # a weight of odd sizes brought to 8 bits
        {"name": "quant_weight_f32", "op": "quant_rows", "type": "f32", "rows": 5000, "D": 2050},
        # one stream's next token: latency, the weights' bytes
        {"name": "ffn_token_bf16", "op": "ffn", "type": "bf16", "M": 1, "K": 2048, "F": 8192, "act": "silu"},
        # a decode batch on 8-bit weights
        {"name": "ffn_batch_e4m3", "op": "ffn", "type": "e4m3", "M": 64, "K": 4096, "F": 8192, "act": "silu"},
        # a prefill on 8-bit weights
        {"name": "ffn_prefill_e4m3", "op": "ffn", "type": "e4m3", "M": 8192, "K": 4096, "F": 8192, "act": "silu"},
        # a training step in float32 with odd sizes
        {"name": "ffn_train_odd_f32", "op": "ffn_train", "type": "f32", "M": 333, "K": 1111, "F": 777, "act": "gelu"},
        # a training step's layer
        {"name": "ffn_train_bf16", "op": "ffn_train", "type": "bf16", "M": 8192, "K": 4096, "F": 8192, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rec", "rec_train", "rec_step", "quant", "quant", "quant_rows", "ffn", "ffn", "ffn", "ffn_train", "ffn_train"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("quant", "quant_rows"):
        D = _log(rng, 40, 8192)
        case = {"op": op, "type": kind, "rows": min(_log(rng, 1, 16384), 16384 * 4096 // D), "D": D}
        return case | ({"res": rng.random() < 0.7} if op == "quant" else {})
    if op in ("ffn", "ffn_train"):
        if op == "ffn":
            kind = rng.choice([kind, "e4m3"])
        M, K, F = _log(rng, 1, 8192), _log(rng, 40, 4096), _log(rng, 40, 8192)
        if rng.random() < 0.6:      # most models' widths are round
            K, F = -(-K // 64) * 64, -(-F // 64) * 64
        if kind == "f32":
            M = min(M, 2048)
        return {"op": op, "type": kind, "M": M, "K": K, "F": F, "act": rng.choice(["silu", "silu", "gelu", "sigmoid", "none"])}
    case = {"op": op, "type": kind, "gtype": rng.choice(["f32", kind])}
    act = rng.choice(["none", "sigmoid", "silu"])
    if op == "rec_step":
        B = _log(rng, 1, 256)
        return case | {"B": B, "T": rng.choice([1, 1, 1, 2, 3]), "D": _log(rng, 40, 4096), "act": act, "pool": B + rng.randint(0, 40)}
    T, D = _log(rng, 1, 16384), _log(rng, 40, 4096)
    nseq = rng.choice([0, 0, rng.randint(1, 24)])
    return case | {"B": 1 if nseq else max(1, min(rng.randint(1, 4), 16384 // T)), "T": T, "D": D, "act": act, "nseq": nseq}


def _lengths(case):
    """The lengths of a packed case's sequences: odd ones, short ones and now and then an empty one."""
    rng = random.Random("%d %d" % (case["T"], case["nseq"]))
    cuts = sorted(rng.randint(0, case["T"]) for _ in range(case["nseq"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    ty = TYPES.get(case["type"])

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] in ("quant", "quant_rows"):
        R, D = case["rows"], case["D"]
        if case["op"] == "quant_rows":
            return s | {"x": (0.02 * rnd(R, D)).to(ty)}
        # a residual stream with a few large channels, as trained models have them
        s["x"] = (rnd(R, D) * (1 + 9 * (torch.rand(D, generator=gen, device="cuda") < 0.01))).to(ty)
        s["r"] = rnd(R, D).to(ty) if case["res"] else None
        return s | {"w": (1 + 0.2 * rnd(D)).to(ty)}
    if case["op"] in ("ffn", "ffn_train"):
        M, K, F = case["M"], case["K"], case["F"]
        x, wg, wu = rnd(M, K), rnd(F, K) * K ** -0.5, rnd(F, K) * K ** -0.5
        if ty is None:      # what a norm with an 8-bit output and a quantised checkpoint leave
            (s["x"], s["sx"]), (s["wg"], s["sg"]), (s["wu"], s["su"]) = _rounded(x), _rounded(wg), _rounded(wu)
            return s
        s |= {"x": x.to(ty), "wg": wg.to(ty), "wu": wu.to(ty)}
        if case["op"] == "ffn_train":
            s["dh"] = (0.1 * rnd(M, F)).to(ty)
        return s
    B, T, D = (case[k] for k in ("B", "T", "D"))
    s["x"] = rnd(B, T, D).to(ty)
    # log decays from gentle to strong, and one in 50 that all but forgets
    g = -torch.nn.functional.softplus(rnd(B, T, D) * 1.5 - 3)
    g -= 20.0 * (torch.rand(B, T, D, generator=gen, device="cuda") < 0.02)
    s["g"] = g.to(TYPES[case["gtype"]])
    s["z"] = None if case["act"] == "none" else rnd(B, T, D).to(ty)
    if case["op"] == "rec_step":
        s["state"] = 0.5 * rnd(case["pool"], D)
        slots = torch.randperm(case["pool"], generator=gen, device="cuda")[:B].to(torch.int32)
        if B > 8:
            slots[torch.randint(B, (B // 16,), generator=gen, device="cuda")] = -1      # idle streams
        return s | {"slots": slots}
    s["cu"] = None
    if case["nseq"]:
        s["cu"] = torch.tensor([0] + _lengths(case), device="cuda").cumsum(0).to(torch.int32)
    s["h0"] = 0.5 * rnd(case["nseq"] or B, D)
    if case["op"] == "rec_train":
        s["dy"] = (0.1 * rnd(B, T, D)).to(ty)
        s["dh"] = 0.1 * rnd(case["nseq"] or B, D)
    return s


def run(s):
    case = s["case"]
    op, act = case["op"], case.get("act")
    if own:
        import deterministic_fp32_gemm_amd as g
        if op == "rec":
            return g.glr_forward(s["x"], s["g"], s["z"], act=act, initial_state=s["h0"], cu_seqlens=s["cu"])[:2]
        if op == "rec_train":
            y, h, marks = g.glr_forward(s["x"], s["g"], s["z"], act=act, initial_state=s["h0"], cu_seqlens=s["cu"])
            return y, h, g.glr_backward(s["x"], s["g"], s["z"], s["dy"], marks, act=act, initial_state=s["h0"], dfinal_state=s["dh"], cu_seqlens=s["cu"])
        if op == "rec_step":
            return g.glr_step(s["x"], s["g"], s["z"], s["state"], act=act, slots=s["slots"]), s["state"]
        if op == "quant":
            return g.norm_quant(s["x"], s["r"], s["w"], eps=EPS)
        if op == "quant_rows":
            return g.quant_rows(s["x"])
        if op == "ffn_train":
            h, kept = g.ffn_forward(s["x"], s["wg"], s["wu"], act=act, keep=True)
            return h, g.ffn_backward(s["dh"], s["x"], s["wg"], s["wu"], kept, act=act)
        if case["type"] == "e4m3":
            return g.ffn_forward(s["x"], s["wg"], s["wu"], act=act, x_scale=s["sx"], gate_scale=s["sg"], up_scale=s["su"])
        return g.ffn_forward(s["x"], s["wg"], s["wu"], act=act)
    return {"rec": _rec_plain, "rec_train": _rec_train_plain, "rec_step": _rec_step_plain, "quant": _quant_plain,
            "quant_rows": lambda s: _rounded(s["x"]), "ffn": _ffn_plain, "ffn_train": _ffn_train_plain}[op](s)


# ---- plain forms: 32 bits, elementary operations --------------------------------------------------------------------
def _act(z, act):
    """act(z) and act'(z)."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    p = 1 / (1 + torch.exp(-z))
    return (p, p * (1 - p)) if act == "sigmoid" else (z * p, p * (1 + z * (1 - p)))


def _gate(s):
    return (1.0, None) if s["z"] is None else _act(s["z"].float(), s["case"]["act"])


def _runs(s):
    """Each run's first and last token among all tokens, and which runs have any."""
    B, T, _ = s["x"].shape
    cu = torch.arange(B + 1, device="cuda") * T if s["cu"] is None else s["cu"].long()
    live = cu[1:] > cu[:-1]
    return cu[:-1][live], cu[1:][live] - 1, live


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 0, by doubling."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _rec_states(s):
    """Decays, states and, before each token, the state it meets; the state after each run."""
    first, last, live = _runs(s)
    x, a = s["x"].flatten(0, 1).to(torch.float32, copy=True), s["g"].flatten(0, 1).float().exp()
    x[first] += a[first] * s["h0"][live]
    cut = a.clone()
    cut[first] = 0
    h = _scan(cut, x)
    met = torch.cat([h[:1], h[:-1]])
    met[first] = s["h0"][live]
    final = s["h0"].clone()
    final[live] = h[last]
    return a, h, met, final


def _rec_plain(s):
    _, h, _, final = _rec_states(s)
    y = h.reshape(s["x"].shape) * _gate(s)[0]
    return y.to(s["x"].dtype), final


def _rec_train_plain(s):
    first, last, live = _runs(s)
    a, h, met, final = _rec_states(s)
    shape, ty = s["x"].shape, s["x"].dtype
    f, df = _gate(s)
    dy = s["dy"].float()
    d = (dy * f).reshape(h.shape)
    d[last] += s["dh"][live]
    after = torch.cat([a[1:], a[:1]])      # the decay that the next token brings, none after a run's last
    after[last] = 0
    d = _scan(after.flip(0), d.flip(0)).flip(0)
    dh0 = s["dh"].clone()
    dh0[live] = a[first] * d[first]
    dz = None if df is None else (dy * h.reshape(shape) * df).to(ty)
    return (h.reshape(shape) * f).to(ty), final, (d.reshape(shape).to(ty), (d * a * met).reshape(shape).to(s["g"].dtype), dz, dh0)


def _rec_step_plain(s):
    live = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    h, out = s["state"][at], []
    for t in range(s["x"].shape[1]):
        h = s["g"][:, t].float().exp() * h + s["x"][:, t].float()
        out.append(h)
    y = torch.stack(out, 1) * _gate(s)[0] * live[:, None, None]
    s["state"][at[live]] = h[live]
    return y.to(s["x"].dtype), s["state"]


def _rounded(y):
    """Rows in 8 bits with their scales."""
    y = y.float()
    scale = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    return (y / scale[..., None]).clamp(-448, 448).to(E4M3), scale


def _quant_plain(s):
    x = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    f = x.float()
    q, scale = _rounded(f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["w"].float())
    return q, scale, x


def _ffn_operands(s):
    x, wg, wu = (s[k].float() for k in ("x", "wg", "wu"))
    return (x * s["sx"][:, None], wg * s["sg"][:, None], wu * s["su"][:, None]) if "sx" in s else (x, wg, wu)


def _ffn_plain(s):
    x, wg, wu = _ffn_operands(s)
    h = _act(x @ wg.t(), s["case"]["act"])[0] * (x @ wu.t())
    return h.to(torch.bfloat16 if "sx" in s else s["x"].dtype)


def _ffn_train_plain(s):
    x, wg, wu = _ffn_operands(s)
    ty = s["x"].dtype
    u, dh = x @ wu.t(), s["dh"].float()
    f, df = _act(x @ wg.t(), s["case"]["act"])
    dg, du = dh * u * df, dh * f
    return (f * u).to(ty), ((dg @ wg + du @ wu).to(ty), (dg.t() @ x).to(ty), (du.t() @ x).to(ty))


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        out = {"rec": _exact_rec, "rec_train": _exact_rec, "rec_step": _exact_step, "quant": _exact_quant, "quant_rows": _exact_quant, "ffn": _exact_ffn, "ffn_train": _exact_ffn}[case["op"]](s)
    return out


def _act64(z, act):
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z if act == "none" else torch.sigmoid(z) * (z if act == "silu" else 1)


def _exact_rec(s):
    """Token by token, all sequences side by side; one that has ended stands still. The gradient goes back through it."""
    B, T, D = s["x"].shape
    if s["cu"] is None:
        first, many = [b * T for b in range(B)], [T] * B
    else:
        c = s["cu"].tolist()
        first, many = c[:-1], [b - a for a, b in zip(c, c[1:])]
    n, longest = len(first), max(many)
    at = torch.tensor(first, device="cuda")[:, None] + torch.arange(longest, device="cuda")
    on = torch.arange(longest, device="cuda") < torch.tensor(many, device="cuda")[:, None]
    at = torch.where(on, at, 0)

    def lay(x):
        return torch.where(on[..., None], x.reshape(B * T, D)[at].double(), 0.0).transpose(0, 1)       # [longest, n, D]

    def back(x):
        out = torch.zeros(B * T, D, dtype=torch.float64, device="cuda")
        out[at[on]] = x.transpose(0, 1)[on]
        return out.reshape(B, T, D)

    x, a = lay(s["x"]), lay(s["g"]).exp()
    met, h = torch.empty(longest + 1, n, D, dtype=torch.float64, device="cuda"), s["h0"].double()
    for t in range(longest):
        met[t] = h
        h = torch.addcmul(x[t], a[t], h)      # past a run's end x is 0 and a is 1
    met[longest] = h
    f = 1.0
    if s["z"] is not None:
        z = s["z"].double().requires_grad_()
        f = _act64(z, s["case"]["act"])
        df, = torch.autograd.grad(f.sum(), z) if "dy" in s else (None,)
        f = f.detach()
    states = back(met[1:])
    if "dy" not in s:
        return states * f, h
    dy = s["dy"].double()
    d, e = lay(dy * f), s["dh"].double()
    for t in reversed(range(longest)):
        d[t] += e
        e = a[t] * d[t]
    dz = None if s["z"] is None else dy * states * df
    return states * f, h, (back(d), back(d * a * met[:longest]), dz, e)


def _exact_step(s):
    state = s["state"].double()
    use = torch.nonzero(s["slots"] >= 0)[:, 0]
    h, y = state[s["slots"][use].long()], torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for t in range(s["x"].shape[1]):
        h = torch.addcmul(s["x"][use, t].double(), torch.exp(s["g"][use, t].double()), h)
        y[use, t] = h if s["z"] is None else h * _act64(s["z"][use, t].double(), s["case"]["act"])
    state[s["slots"][use].long()] = h
    return y, state


def _exact_quant(s):
    x = s["x"].double()
    if s["case"]["op"] == "quant_rows":
        scale = (x.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
        return x / scale[:, None], scale
    x = x if s["r"] is None else x + s["r"].double()
    kept = x.to(s["x"].dtype).double()
    y = kept / (kept.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w"].double()
    scale = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    return y / scale[:, None], scale, x


def _exact_ffn(s):
    """Differentiated by machine from the definition."""
    x, wg, wu = ((s[k].double() * (s[c].double()[:, None] if c in s else 1)).requires_grad_("dh" in s) for k, c in (("x", "sx"), ("wg", "sg"), ("wu", "su")))
    h = _act64(torch.nn.functional.linear(x, wg), s["case"]["act"]) * torch.nn.functional.linear(x, wu)
    if "dh" not in s:
        return h
    return h.detach(), torch.autograd.grad(h, (x, wg, wu), s["dh"].double())


def work(case):
    t = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}[case["type"]]
    op = case["op"]
    if op in ("quant", "quant_rows"):
        n, res = case["rows"] * case["D"], case.get("res", False)
        arrays = (3 if res else 1) if op == "quant" else 1      # x, with a residual that and x'
        return {"bytes": n * (arrays * t + 1) + 4 * case["rows"] + (case["D"] * t if op == "quant" else 0), "flops": 8 * n}
    if op in ("ffn", "ffn_train"):
        M, K, F = (case[k] for k in ("M", "K", "F"))
        out = 2 if case["type"] == "e4m3" else t
        ends = (M * K + 2 * F * K) * t
        if op == "ffn":
            return {"bytes": ends + M * F * out + (4 * (M + 2 * F) if t == 1 else 0), "flops": 4 * M * K * F}
        return {"bytes": 2 * ends + 2 * M * F * t, "flops": 12 * M * K * F}
    n, gt, z = case["B"] * case["T"] * case["D"], TYPES[case["gtype"]].itemsize, case["act"] != "none"
    if op == "rec_step":
        live = case["B"] - (case["B"] // 16 if case["B"] > 8 else 0)
        return {"bytes": n * (2 * t + gt + z * t) + 8 * live * case["D"], "flops": 8 * n}
    states = 8 * (case["nseq"] or case["B"]) * case["D"]
    forward = n * (2 * t + gt + z * t) + states
    if op == "rec":
        return {"bytes": forward, "flops": 8 * n}
    # x, g, z and dy read once, y, dx, dg and dz written once
    return {"bytes": forward + n * (2 * t + gt + z * t) + states, "flops": 30 * n}
