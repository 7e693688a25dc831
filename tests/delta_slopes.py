"""Gradients of a model's parameters against differences of its loss, one parameter at a time along its own gradient, where
the slope is the gradient's norm: a gradient that is zero, of the wrong sign, or no more than partly right shows."""

import torch


def slope_errors(params, loss_of, h):
    """|difference / slope - 1| of each named parameter, from central differences of step h; inf where the gradient is zero
    or missing. The parameters are as before afterwards."""
    for p in params.values():
        p.grad = None
    loss_of().backward()
    errors = {}
    for name, p in params.items():
        norm = 0.0 if p.grad is None else float(p.grad.double().norm())
        if norm == 0.0:
            errors[name] = float("inf")
            continue
        keep, way = p.detach().clone(), p.grad / norm
        ends = []
        with torch.no_grad():
            for s in (1, -1):
                p.copy_(keep + s * h * way)
                ends.append(float(loss_of()))
            p.copy_(keep)
        errors[name] = abs((ends[0] - ends[1]) / (2 * h) / norm - 1)
    return errors
