"""The delta entry points in torch's graph: what gdr_forward, norm_forward and gdr_step go through when a tensor of the call
requires a gradient and grad mode is on. The gradients are gdr_backward's and norm_backward's, once differentiable."""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import delta


class GatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_state, scale, final_state, cu_seqlens):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_seqlens)
        ctx.scale = scale
        return delta.gdr_forward(q, k, v, g, beta, scale=scale, initial_state=initial_state, final_state=final_state,
                                 cu_seqlens=cu_seqlens)

    @staticmethod
    @once_differentiable
    def backward(ctx, do, ds):
        q, k, v, g, beta, initial_state, cu_seqlens = ctx.saved_tensors
        if do is None:          # only the last state was used
            do = torch.zeros_like(v)
        *grads, ds0 = delta.gdr_backward(q, k, v, g, beta, do, scale=ctx.scale, initial_state=initial_state,
                                         dfinal_state=ds, cu_seqlens=cu_seqlens)
        return (*grads, None if initial_state is None else ds0, None, None, None)


class BlockNorm(torch.autograd.Function):
    """(x_new, y, rstd); without o, whose call's x_new is x itself, (y, rstd)."""

    @staticmethod
    def forward(ctx, x, o, z, w_post, w_pre, scale, act, eps):
        ctx.set_materialize_grads(False)
        x_new, y, rstd = delta.norm_forward(x, o, z, w_post, w_pre, scale, act=act, eps=eps)
        ctx.save_for_backward(x_new, o, z, w_post, w_pre, scale, rstd)
        ctx.act, ctx.has_x = act, x is not None
        ctx.mark_non_differentiable(rstd)
        return (y, rstd) if o is None else (x_new, y, rstd)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        x_new, o, z, w_post, w_pre, scale, rstd = ctx.saved_tensors
        dx_new, dy = (None, grads[0]) if o is None else grads[:2]
        if dy is None and dx_new is None:
            return (None,) * 8
        if dy is None:          # y was not used: the second norm has no part
            w_pre = None
        dx, do, dz, dw_post, dw_pre, dscale = delta.norm_backward(dx_new, dy, x_new, o, z, w_post, w_pre, scale, rstd,
                                                                  act=ctx.act)
        return dx if ctx.has_x else None, do, dz, dw_post, dw_pre, dscale, None, None


class NoGradient(torch.autograd.Function):
    """`made`'s one tensor, an output of what has no gradient: a backward pass that reaches it is an error."""

    @staticmethod
    def forward(ctx, made, name, *inputs):
        ctx.name = name
        return made[0]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no gradient: call it under torch.no_grad(), or use gdr_forward")
