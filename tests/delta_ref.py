"""The gated delta rule and the block norm in float64 on the CPU, straight from their definitions: the recurrence token
by token, gradients by automatic differentiation of it. Shares nothing with the kernels."""

import torch


def gdr(q, k, v, g, beta, scale, s0=None, cu=None):
    """(o, final states) in float64; tensors of any float type and device."""
    q, k, v, g, beta = (t.double() if t.dtype != torch.float64 else t for t in (q, k, v, g, beta))
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    q, k = (t.repeat_interleave(Hv // Hk, 2) for t in (q, k))
    runs = [(b, 0, T) for b in range(B)] if cu is None else [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]
    o = [[torch.zeros(Hv, dv, dtype=torch.float64) for _ in range(T)] for _ in range(B)]
    final = []
    for i, (b, lo, hi) in enumerate(runs):
        S = torch.zeros(Hv, dk, dv, dtype=torch.float64) if s0 is None else s0[i].double()
        for t in range(lo, hi):
            S = S * torch.exp(g[b, t])[:, None, None]
            u = beta[b, t][:, None] * (v[b, t] - torch.einsum("hk,hkv->hv", k[b, t], S))
            S = S + k[b, t][:, :, None] * u[:, None, :]
            o[b][t] = scale * torch.einsum("hk,hkv->hv", q[b, t], S)
        final.append(S)
    o = torch.stack([torch.stack(x) for x in o]) if T else torch.zeros(B, 0, Hv, dv, dtype=torch.float64)
    return o, torch.stack(final)


def gdr_grads(q, k, v, g, beta, do, scale, s0=None, ds=None, cu=None):
    """Gradients of q, k, v, g, beta, s0 in float64."""
    n = (len(cu) - 1) if cu is not None else q.shape[0]
    state = torch.zeros(n, v.shape[2], q.shape[3], v.shape[3], dtype=torch.float64) if s0 is None else s0.double()
    leaves = [t.double().clone().requires_grad_() for t in (q, k, v, g, beta)] + [state.clone().requires_grad_()]
    o, S = gdr(*leaves[:5], scale, leaves[5], cu)
    total = (o * do.double()).sum()
    if ds is not None:
        total = total + (S * ds.double()).sum()
    return torch.autograd.grad(total, leaves)


def act(z, kind):
    return 1.0 if kind == "none" else torch.sigmoid(z) * (z if kind == "silu" else 1.0)


def norm(x, o, z, w_post, w_pre, scale, kind, eps, stored):
    """(x_new, y, rstd) in float64; y is that of x_new rounded to `stored`."""
    r1 = r2 = None
    xn = x.double() if x is not None else 0.0
    if o is not None:
        o = o.double()
        r1 = 1 / (o.square().mean(-1, keepdim=True) + eps).sqrt()
        xn = xn + scale.double() * (o * r1 * w_post.double()) * act(None if z is None else z.double(), kind)
    y = None
    if w_pre is not None:
        kept = xn.to(stored).double()
        r2 = 1 / (kept.square().mean(-1, keepdim=True) + eps).sqrt()
        y = kept * r2 * w_pre.double()
    return xn, y, r1, r2


def norm_grads(dxn, dy, xn, o, z, w_post, w_pre, scale, kind, eps):
    """(dx, do, dz, dw_post, dw_pre, dscale) in float64 at the stored x_new; None where there is none."""
    leaf = lambda t: None if t is None else t.double().clone().requires_grad_()  # noqa: E731
    dw2, dx = None, 0.0 if dxn is None else dxn.double()
    if w_pre is not None:
        x, w = leaf(xn), leaf(w_pre)
        y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
        gx, dw2 = torch.autograd.grad(y, (x, w), dy.double())
        dx = dx + gx
    if o is None:
        return dx, None, None, None, dw2, None
    o, z, w, s = leaf(o), leaf(z), leaf(w_post), leaf(scale)
    add = s * (o / (o.square().mean(-1, keepdim=True) + eps).sqrt() * w) * act(z, kind)
    got = torch.autograd.grad(add, [t for t in (o, w, s, z) if t is not None], dx)
    return dx, got[0], got[3] if z is not None else None, got[1], dw2, got[2]
