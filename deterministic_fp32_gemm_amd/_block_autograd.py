"""The entry points of block.py in torch's graph: what glr_forward, ffn_forward and those without a gradient go through when
a tensor of the call requires one and grad mode is on. The gradients are glr_backward's and ffn_backward's, once
differentiable."""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import block


class GatedLinearRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, z, initial_state, act, cu_seqlens):
        ctx.set_materialize_grads(False)
        y, h, marks = block.glr_forward(x, g, z, act=act, initial_state=initial_state, cu_seqlens=cu_seqlens)
        ctx.save_for_backward(x, g, z, initial_state, cu_seqlens, marks)
        ctx.act = act
        ctx.mark_non_differentiable(marks)
        return y, h, marks

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh, _):
        x, g, z, initial_state, cu_seqlens, marks = ctx.saved_tensors
        if dy is None:
            if dh is None:
                return (None,) * 6
            dy = torch.zeros_like(x)        # only the last state was used
        dx, dg, dz, dh0 = block.glr_backward(x, g, z, dy, marks, act=ctx.act, initial_state=initial_state, dfinal_state=dh,
                                             cu_seqlens=cu_seqlens)
        return dx, dg, dz, None if initial_state is None else dh0, None, None


class GatedFeedForward(torch.autograd.Function):
    """(h, g, u); the products are not differentiable outputs."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, act, precise):
        ctx.set_materialize_grads(False)
        h, kept = block.ffn_forward(x, w_gate, w_up, act=act, keep=True)
        ctx.save_for_backward(x, w_gate, w_up, *kept)
        ctx.act, ctx.precise = act, precise
        ctx.mark_non_differentiable(*kept)
        return (h, *kept)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, *_):
        if dh is None:
            return (None,) * 5
        x, w_gate, w_up, *kept = ctx.saved_tensors
        return (*block.ffn_backward(dh, x, w_gate, w_up, kept, act=ctx.act, precise=ctx.precise), None, None)


class NoGradient(torch.autograd.Function):
    """`made`'s one tensor, an output of what has no gradient: a backward pass that reaches it is an error."""

    @staticmethod
    def forward(ctx, made, name, *inputs):
        ctx.name = name
        return made[0]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no gradient: call it under torch.no_grad()")
