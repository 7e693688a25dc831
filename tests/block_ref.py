"""References in 64 bits for the operators of libsdm_block, each with a bound on what float32 arithmetic and the output's
rounding may be off by, element by element."""

import math

import torch

U = 2.0 ** -24          # half a step of float32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half(ty):
    """The largest relative error of one rounding to ty."""
    return torch.finfo(ty).eps / 2


def tiny(ty):
    """Half the smallest step of ty."""
    return torch.finfo(ty).smallest_normal * torch.finfo(ty).eps / 2


def act64(z, act):
    """act(z), act'(z) and a bound of |act''|."""
    if act == "none":
        return z, torch.ones_like(z), 0.0
    if act == "gelu":
        p, e = torch.special.ndtr(z), torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return z * p, p + z * e, 0.8        # |2 e - z^2 e| <= 2 / sqrt(2 pi)
    p, q = torch.sigmoid(z), torch.sigmoid(-z)
    return (p, p * q, 0.1) if act == "sigmoid" else (z * p, p * (1 + z * q), 0.5)


# What act or act' of a float32 may be off by, relative to 1 + |z|: e^-|z| carries an argument rounded to 2^-24 (its error is
# at most |z| 2^-23 e^-|z| < 2^-23 in all), and four more operations follow; the hardware's exponential and reciprocal are
# within 2^-23, the library's closer. erfc is within 4 steps of its own, which z multiplies.
GATE = 16 * U


def within(got, want, bound, what=""):
    got, want, bound = got.double().cpu(), want.cpu(), bound.cpu()
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()}, by up to {float((off / bound).max()):.3g} times the bound, "
                           f"at {tuple(torch.nonzero(bad)[0].tolist())}")


def runs_of(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def glr(x, g, z, act, h0, cu=None, dy=None, dh=None):
    """{name: (value, bound)} of the gated linear recurrence's outputs, and with dy of its gradient. CPU, token by token.

    A step h = a h + x in float32 is off by 2^-24 |h| (the fused sum) and a |h_prev| times what a is off by: 2^-23 for the
    exponential, and 2^-24 for each product by which A is composed. Tokens go through at most one composition a wavefront, one
    a tile and one a part, each another rounding of A, of H and of the sum: 8 roundings a step cover them. With m the same
    recurrence over |x|, which bounds |h|, the error e obeys e_t <= a e_{t-1} + 8 2^-24 m_t."""
    B, T, D = x.shape
    ty, runs = x.dtype, runs_of(B, T, cu)
    X, A = x.double().cpu(), g.double().cpu().exp()
    H0 = torch.zeros(len(runs), D, dtype=torch.float64) if h0 is None else h0.double().cpu()
    Z = None if z is None else z.double().cpu()
    f, df, _ = (1.0, None, 0) if z is None else act64(Z, act)
    gate = 0.0 if z is None else GATE * (1 + Z.abs())
    h, m, e, met, emet = (torch.zeros(B, T, D, dtype=torch.float64) for _ in range(5))
    last, elast = H0.clone(), torch.zeros_like(H0)
    for i, (b, s, t1) in enumerate(runs):
        c, mm, ee = H0[i], H0[i].abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(s, t1):
            met[b, t], emet[b, t] = c, ee
            c, mm = A[b, t] * c + X[b, t], A[b, t] * mm + X[b, t].abs()
            ee = A[b, t] * ee + 8 * U * mm
            h[b, t], m[b, t], e[b, t] = c, mm, ee
        last[i], elast[i] = c, ee
    y = h * f
    fa = 1.0 if z is None else f.abs()
    out = {"y": (y, half(ty) * y.abs() * 1.01 + 1.01 * (e * fa + h.abs() * gate + U * y.abs()) + tiny(ty)),
           "state": (last, elast + 1e-40)}
    if dy is None:
        return out
    DY = dy.double().cpu()
    DH = torch.zeros_like(H0) if dh is None else dh.double().cpu()
    v = DY * f
    ev = DY.abs() * gate + U * v.abs()
    d, ed = torch.zeros_like(h), torch.zeros_like(h)
    dh0, edh0 = DH.clone(), torch.zeros_like(DH)
    for i, (b, s, t1) in enumerate(runs):
        c, mm, ee = DH[i], DH[i].abs(), torch.zeros(D, dtype=torch.float64)
        for t in reversed(range(s, t1)):
            c, mm = v[b, t] + c, v[b, t].abs() + mm
            ee = ee + ev[b, t] + 8 * U * mm
            d[b, t], ed[b, t] = c, ee
            c, mm, ee = A[b, t] * c, A[b, t] * mm, A[b, t] * ee
        dh0[i], edh0[i] = c, ee + 4 * U * mm
    gt = g.dtype
    dg = d * A * met
    edg = A * (ed * met.abs() + d.abs() * emet + ed * emet) + 6 * U * dg.abs()
    out["dx"] = (d, half(ty) * d.abs() * 1.01 + 1.01 * ed + tiny(ty))
    out["dg"] = (dg, half(gt) * dg.abs() * 1.01 + 1.01 * edg + tiny(gt))
    out["dh0"] = (dh0, edh0 + 1e-40)
    if z is not None:
        dz = DY * h * df
        out["dz"] = (dz, half(ty) * dz.abs() * 1.01 + 1.01 * DY.abs() * (e * df.abs() + h.abs() * gate + 2 * U * (h * df).abs()) + tiny(ty))
    return out


def cut8(X, W):
    """What the matrix cores' 8-bit products may lose. The instruction aligns the products of 8 adjacent elements and cuts each
    off, towards zero, below 2^-13 of 2^e, e the largest sum of two exponents among them: beside 2^8 2^8 a product of 2^3 is
    kept and one of 7/8 2^3 is not. 2^e is at most the largest product p, which itself keeps its 8 bits, so a group loses less
    than 7 2^-13 max |p|. (The sums of groups meet the accumulator with float32's 24 bits.)"""
    lost = torch.zeros(X.shape[0], W.shape[0], dtype=torch.float64, device=X.device)
    for k in range(0, X.shape[1], 8):
        lost += (X[:, None, k:k + 8] * W[None, :, k:k + 8]).abs().amax(-1)
    return 7 * 2.0 ** -13 * lost


def ffn(x, wg, wu, act, otype, scales=(None, None, None), dh=None, parts=1):
    """{name: (value, bound)} of the gated feed-forward product, and with dh of its gradient. On x's device.

    A sum of K products in float32 is off by at most (K + 8) 2^-23 of the sum of their absolute values (a rounding or a cut-off
    for each of them, and for what joins the parts of the sum); float32 operands in parts leave out less than 2^-23 of a
    product and round the joined parts as often."""
    X, G, W = (t.double() if s is None else t.double() * s.double()[:, None] for t, s in zip((x, wg, wu), scales))
    K, F, M = X.shape[1], G.shape[0], X.shape[0]
    # the scales are applied to the finished sum, with two roundings
    eps = lambda n: 2 * (n + 8) * U * (6 if x.dtype == torch.float32 else 1) + 4 * U  # noqa: E731
    g, u = X @ G.t(), X @ W.t()
    eg, eu = eps(K) * (X.abs() @ G.abs().t()), eps(K) * (X.abs() @ W.abs().t())
    if scales[0] is not None:
        eg, eu = eg + cut8(X, G), eu + cut8(X, W)
    f, df, dd = act64(g, act)
    gate = GATE * (1 + g.abs())
    ef = gate + (df.abs() + dd * eg) * eg
    h = f * u
    out = {"h": (h, half(otype) * h.abs() * 1.01 + 1.01 * (ef * u.abs() + (f.abs() + ef) * eu + U * h.abs()) + tiny(otype)),
           "g": (g, eg + tiny(torch.float32)), "u": (u, eu + tiny(torch.float32))}
    if dh is None:
        return out
    ty, DH = x.dtype, dh.double()
    edf = gate + dd * eg * (1 + (1 if act == "none" else 2) * eg)
    dg, du = DH * u * df, DH * f
    rough = half(ty) ** parts if ty != torch.float32 else 4 * U     # dg and du as the products take them
    # a value under the type's range rounds to a multiple of its smallest step
    edg = DH.abs() * (eu * (df.abs() + edf) + u.abs() * edf) + (rough + 2 * U) * dg.abs() * 1.01 + tiny(ty)
    edu = DH.abs() * ef + (rough + 2 * U) * du.abs() * 1.01 + tiny(ty)
    for name, v, e, n in (("dx", dg @ G + du @ W, edg @ G.abs() + edu @ W.abs() + eps(2 * F) * (dg.abs() @ G.abs() + du.abs() @ W.abs()), F),
                          ("dwg", dg.t() @ X, edg.t() @ X.abs() + eps(M) * (dg.abs().t() @ X.abs()), M),
                          ("dwu", du.t() @ X, edu.t() @ X.abs() + eps(M) * (du.abs().t() @ X.abs()), M)):
        out[name] = (v, half(ty) * v.abs() * 1.01 + 1.01 * e + tiny(ty))
    return out


def e4m3_step(v):
    """The distance between neighbours of e4m3 at |v|."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
