"""The feed-forward half of a transformer layer over the operators of layer.py.

``FeedForward`` is the pre-norm block ``s + W2 act(W1 norm(s) + b1) + b2`` with
``s = x + residual``; ``ExpertsFeedForward`` replaces the two linears by each
token's chosen experts, weighted by its router.  Both return the new residual
stream, so that blocks chain with the norm's own addition, and train through
the autograd functions here, whose every step is a libmc2 call: the only torch
operations are views and the router's choice (a top-k and a softmax).  Their
gradients cannot be differentiated again: a second backward through them raises.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._autograd import first_order
from .layer import (MC2_ACT_GELU, MC2_ACT_NONE, MC2_ACT_SILU, mc2_add_rms_norm, mc2_add_rms_norm_grad, mc2_linear_act,
                    mc2_linear_act_grad, mc2_moe_permute, mc2_moe_unpermute, mc2_moe_unpermute_grad)

__all__ = ["AddRMSNormFunction", "LinearActFunction", "PermuteFunction", "UnpermuteFunction", "FeedForward",
           "ExpertsFeedForward"]


def _ready(grad):
    """An incoming gradient as the library takes it: contiguous and 16-byte aligned (one that is a part of a
    concatenation's may start anywhere)."""
    grad = grad.contiguous()
    return grad.clone() if grad.data_ptr() % 16 else grad


class AddRMSNormFunction(torch.autograd.Function):
    """(norm(x + residual) * weight, x + residual)."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps: float):
        out, _, s, rstd = mc2_add_rms_norm(x, weight, residual, eps=eps, need_rstd=True)
        ctx.save_for_backward(s, weight, rstd)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)  # no zeros for a stream that ends here
        # without a residual the sum is x itself, which a function may not return as its output
        return out, s if ctx.has_residual else s.view_as(s)

    @staticmethod
    @first_order
    def backward(ctx, dout, dsum):
        s, weight, rstd = ctx.saved_tensors
        if dout is None:
            return dsum, dsum if ctx.has_residual else None, None, None
        dx, dweight = mc2_add_rms_norm_grad(_ready(dout), s, weight, rstd, None if dsum is None else _ready(dsum))
        return dx, dx if ctx.has_residual else None, dweight, None


class LinearActFunction(torch.autograd.Function):
    """residual + act(x @ w^T + bias), of one matrix or of groups of rows."""

    @staticmethod
    def forward(ctx, x, w, bias, residual, act: int, group_offsets):
        out, z = mc2_linear_act(x, w, bias, residual, act=act, group_offsets=group_offsets,
                                need_z=act != MC2_ACT_NONE)
        ctx.save_for_backward(x, w, z, group_offsets)
        ctx.act, ctx.has_bias, ctx.has_residual = act, bias is not None, residual is not None
        return out

    @staticmethod
    @first_order
    def backward(ctx, dout):
        x, w, z, group_offsets = ctx.saved_tensors
        dout = _ready(dout)
        dx, dw, dbias = mc2_linear_act_grad(dout, x, w, z, act=ctx.act, group_offsets=group_offsets,
                                            need_dx=ctx.needs_input_grad[0], need_dw=ctx.needs_input_grad[1],
                                            need_dbias=ctx.has_bias and ctx.needs_input_grad[2])
        return dx, dw, dbias, dout if ctx.has_residual else None, None, None


class PermuteFunction(torch.autograd.Function):
    """(rows sorted by expert, row_map, offsets)."""

    @staticmethod
    def forward(ctx, x, expert_ids, experts: int):
        out, row_map, offsets = mc2_moe_permute(x, expert_ids, experts)
        ctx.save_for_backward(row_map)
        ctx.mark_non_differentiable(row_map, offsets)
        return out, row_map, offsets

    @staticmethod
    @first_order
    def backward(ctx, dout, _map, _offsets):
        (row_map,) = ctx.saved_tensors
        return mc2_moe_unpermute(_ready(dout), row_map), None, None


class UnpermuteFunction(torch.autograd.Function):
    """The experts' rows summed back in token order with the router's weights."""

    @staticmethod
    def forward(ctx, y, row_map, weights):
        ctx.save_for_backward(y, row_map, weights)
        return mc2_moe_unpermute(y, row_map, weights)

    @staticmethod
    @first_order
    def backward(ctx, dout):
        y, row_map, weights = ctx.saved_tensors
        dy, dweights = mc2_moe_unpermute_grad(_ready(dout), y, row_map, weights,
                                              need_dweights=ctx.needs_input_grad[2])
        return dy, None, dweights


def _param(*shape, std, dtype, device):
    return torch.nn.Parameter(torch.randn(shape, device=device, dtype=torch.float32).mul_(std).to(dtype))


class FeedForward(torch.nn.Module):
    """Pre-norm feed-forward of x (tokens, h): returns s + W2 act(W1 norm(s) + b1) + b2, s = x + residual."""

    def __init__(self, h: int, hidden: int, act: int = MC2_ACT_GELU, eps: float = 1e-6, dtype=torch.bfloat16,
                 device="cuda"):
        super().__init__()
        self.act, self.eps = act, eps
        kw = dict(dtype=dtype, device=device)
        self.norm = torch.nn.Parameter(torch.ones((h,), **kw))
        self.w1, self.b1 = _param(hidden, h, std=h ** -0.5, **kw), torch.nn.Parameter(torch.zeros((hidden,), **kw))
        self.w2, self.b2 = _param(h, hidden, std=hidden ** -0.5, **kw), torch.nn.Parameter(torch.zeros((h,), **kw))

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        y, s = AddRMSNormFunction.apply(x, residual, self.norm, self.eps)
        a = LinearActFunction.apply(y, self.w1, self.b1, None, self.act, None)
        return LinearActFunction.apply(a, self.w2, self.b2, s, MC2_ACT_NONE, None)


class ExpertsFeedForward(torch.nn.Module):
    """Mixture-of-experts feed-forward of x (tokens, h): returns (the experts' weighted sum, s = x + residual),
    which the next block's norm adds.  Each token takes the `top` experts its router scores highest,
    weighted by the softmax over their scores."""

    def __init__(self, h: int, hidden: int, experts: int, top: int, act: int = MC2_ACT_SILU, eps: float = 1e-6,
                 dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.experts, self.top, self.act, self.eps = experts, top, act, eps
        kw = dict(dtype=dtype, device=device)
        self.norm = torch.nn.Parameter(torch.ones((h,), **kw))
        self.router = _param(experts, h, std=h ** -0.5, **kw)
        self.w1 = _param(experts, hidden, h, std=h ** -0.5, **kw)
        self.w2 = _param(experts, h, hidden, std=hidden ** -0.5, **kw)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        y, s = AddRMSNormFunction.apply(x, residual, self.norm, self.eps)
        score = LinearActFunction.apply(y, self.router, None, None, MC2_ACT_NONE, None).float()
        top, ids = score.topk(self.top, dim=-1)
        rows, row_map, offsets = PermuteFunction.apply(y, ids.to(torch.int32), self.experts)
        a = LinearActFunction.apply(rows, self.w1, None, None, self.act, offsets)
        e = LinearActFunction.apply(a, self.w2, None, None, MC2_ACT_NONE, offsets)
        return UnpermuteFunction.apply(e, row_map, torch.softmax(top, dim=-1)), s
