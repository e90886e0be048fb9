"""Backward functions that libmc2 computes, and whose results therefore carry no graph."""
from __future__ import annotations

import functools

import torch


class _FirstOrder(torch.autograd.Function):
    @staticmethod
    def forward(ctx, *grads):
        return tuple(g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("second derivatives through libmc2's operators are not implemented")


def first_order(backward):
    """Decorator of a ``backward``: differentiating its results (``create_graph=True`` and then a second
    backward through them) raises, whatever of ``ctx`` and of the incoming gradients they depend on, where
    autograd would drop their terms without a word.  (``once_differentiable`` does so only if an incoming
    gradient has a graph, which that of a plain sum has not.)"""
    @functools.wraps(backward)
    def wrapper(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        out = list(out) if isinstance(out, tuple) else [out]
        at = [i for i, g in enumerate(out) if g is not None]
        if at:
            for i, g in zip(at, _FirstOrder.apply(*(out[i].detach().requires_grad_() for i in at))):
                out[i] = g
        return tuple(out)

    return wrapper
