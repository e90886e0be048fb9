"""The feed-forward half of a transformer layer over the operators of layer.py.

``FeedForward`` is the pre-norm block ``s + W2 act(W1 norm(s) + b1) + b2`` with
``s = x + residual``; ``ExpertsFeedForward`` replaces the two linears by each
token's chosen experts, weighted by its router.  Both return the new residual
stream, so that blocks chain with the norm's own addition, and train through
the autograd functions here, whose every step is a libmc2 call: the only torch
operations are views and, without a `score`, the router's choice (a top-k and a
softmax).  Their gradients cannot be differentiated again: a second backward
through them raises.  A step is captured into a graph forward and backward
together, while no eager autograd graph of the same parameters lives (its nodes
stay on the stream they were made on, which a capture may not touch).

With `keep8` a block keeps its linears' input and pre-activation for the
backward as int8 codes with a scale per 128 columns, and no activation: per row
h + hidden bytes where it would keep 2 h + 4 hidden.  A dense block has a row
per token; an experts block has `top`, and keeps their experts' output (2 h
bytes a row) and the router's input (2 h a token) besides, with keep8 or
without: top (3 h + hidden) + 2 h bytes a token, where it would keep top (4 h +
4 hidden) + 2 h.  To that come the residual stream and small tensors (scales,
logits, ids, weights).  The forward is the same; the gradients are those at the
codes' values (of a pre-activation that overflowed to -inf, 0, as in 16 bits;
one of +inf, which leaves no finite output, counts as the largest finite of its
128 columns).

``Int8FeedForward`` and ``Int8ExpertsFeedForward`` serve a trained block with
int8 codes for its weights (a scale per output channel) and its activations
(one per token).
"""
from __future__ import annotations

from typing import Optional

import torch

from ._autograd import first_order
from .layer import (MC2_ACT_GELU, MC2_ACT_NONE, MC2_ACT_SILU, mc2_add_rms_norm, mc2_add_rms_norm_grad, mc2_linear_act,
                    mc2_linear_act_grad, mc2_moe_permute, mc2_moe_unpermute, mc2_moe_unpermute_grad)
from .layer8 import mc2_linear_act_grad_i8, mc2_linear_i8, mc2_moe_route, mc2_moe_route_grad, mc2_quant_rows

__all__ = ["AddRMSNormFunction", "LinearActFunction", "KeptLinearsFunction", "RouteFunction", "PermuteFunction",
           "UnpermuteFunction", "FeedForward", "ExpertsFeedForward", "Int8FeedForward", "Int8ExpertsFeedForward"]


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


class KeptLinearsFunction(torch.autograd.Function):
    """residual + act(x @ w1^T + b1) @ w2^T + b2, of one pair of matrices or of groups of rows, whose backward works
    from int8 codes of x and of the pre-activation."""

    @staticmethod
    def forward(ctx, x, w1, b1, w2, b2, residual, act: int, group_offsets):
        kept = any(ctx.needs_input_grad)  # (a frozen block on rows that need no gradient has no backward)
        a, z = mc2_linear_act(x, w1, b1, act=act, group_offsets=group_offsets, need_z=kept)
        out, _ = mc2_linear_act(a, w2, b2, residual, act=MC2_ACT_NONE, group_offsets=group_offsets)
        if not kept:
            return out
        # a pre-activation past its 16 bits' range is an infinity, which is to cost the other columns nothing
        inf = dict(keep_inf=True) if z.element_size() == 2 else {}
        ctx.save_for_backward(*mc2_quant_rows(x, group=128), *mc2_quant_rows(z, group=128, **inf), w1, w2, group_offsets)
        ctx.act, ctx.biases, ctx.has_residual = act, (b1 is not None, b2 is not None), residual is not None
        return out

    @staticmethod
    @first_order
    def backward(ctx, dout):
        x, xs, z, zs, w1, w2, group_offsets = ctx.saved_tensors
        need, dout = ctx.needs_input_grad, _ready(dout)
        first = need[0] or need[1] or (need[2] and ctx.biases[0])
        # the second linear's input is the activation of what was kept
        da, dw2, db2 = mc2_linear_act_grad_i8(dout, z, zs, w2, act=MC2_ACT_NONE, x_act=ctx.act, need_dx=first,
                                              group_offsets=group_offsets, need_dw=need[3],
                                              need_dbias=ctx.biases[1] and need[4])
        dx = dw1 = db1 = None
        if first:
            dx, dw1, db1 = mc2_linear_act_grad_i8(da, x, xs, w1, z, zs, act=ctx.act, group_offsets=group_offsets,
                                                  need_dx=need[0], need_dw=need[1],
                                                  need_dbias=ctx.biases[0] and need[2])
        return dx, dw1, db1, dw2, db2, dout if ctx.has_residual else None, None, None


class RouteFunction(torch.autograd.Function):
    """(each token's experts, their weights) of a router's logits; `kind` is mc2_moe_route's keywords."""

    @staticmethod
    def forward(ctx, logits, bias, top: int, kind: dict):
        ids, weights = mc2_moe_route(logits, top, bias, **kind)
        ctx.save_for_backward(logits, ids)
        ctx.kind = {k: v for k, v in kind.items() if k in ("score", "renormalise", "scale")}
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    @first_order
    def backward(ctx, _ids, dweights):
        logits, ids = ctx.saved_tensors
        return mc2_moe_route_grad(_ready(dweights), logits, ids, **ctx.kind), None, None, None


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
                 device="cuda", keep8: bool = False):
        super().__init__()
        self.act, self.eps, self.keep8 = act, eps, keep8
        kw = dict(dtype=dtype, device=device)
        self.norm = torch.nn.Parameter(torch.ones((h,), **kw))
        self.w1, self.b1 = _param(hidden, h, std=h ** -0.5, **kw), torch.nn.Parameter(torch.zeros((hidden,), **kw))
        self.w2, self.b2 = _param(h, hidden, std=hidden ** -0.5, **kw), torch.nn.Parameter(torch.zeros((h,), **kw))

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        y, s = AddRMSNormFunction.apply(x, residual, self.norm, self.eps)
        if self.keep8 and torch.is_grad_enabled():
            return KeptLinearsFunction.apply(y, self.w1, self.b1, self.w2, self.b2, s, self.act, None)
        a = LinearActFunction.apply(y, self.w1, self.b1, None, self.act, None)
        return LinearActFunction.apply(a, self.w2, self.b2, s, MC2_ACT_NONE, None)


class ExpertsFeedForward(torch.nn.Module):
    """Mixture-of-experts feed-forward of x (tokens, h): returns (the experts' weighted sum, s = x + residual),
    which the next block's norm adds.  Each token takes the `top` experts its router scores highest,
    weighted by the softmax over their scores.

    With a `score` (MC2_SCORE_SOFTMAX or MC2_SCORE_SIGMOID) the choice is mc2_moe_route's: experts in `groups`,
    of which top_groups are kept by the sum of their group_top best, weights renormalised and scaled.  `balance`
    adds the buffer `bias` (experts) fp32 to the scores in the choice alone, for the caller to move.

    A token with a NaN among its logits, or under a softmax one of +inf (past fp16's range), leaves as a row of NaN; one
    whose experts are all off (a bias of -inf) as a row of 0."""

    def __init__(self, h: int, hidden: int, experts: int, top: int, act: int = MC2_ACT_SILU, eps: float = 1e-6,
                 dtype=torch.bfloat16, device="cuda", keep8: bool = False, score: Optional[int] = None,
                 groups: int = 1, top_groups: int = 1, group_top: int = 1, renormalise: bool = True,
                 scale: float = 1.0, balance: bool = False):
        super().__init__()
        self.experts, self.top, self.act, self.eps, self.keep8 = experts, top, act, eps, keep8
        self.kind = None if score is None else dict(score=score, groups=groups, top_groups=top_groups,
                                                    group_top=group_top, renormalise=renormalise, scale=scale,
                                                    keep_nan=True)
        if score is None and (groups, top_groups, group_top, renormalise, scale, balance) != (1, 1, 1, True, 1.0, False):
            raise ValueError("groups, weights and a balancing bias need a score")
        kw = dict(dtype=dtype, device=device)
        self.norm = torch.nn.Parameter(torch.ones((h,), **kw))
        self.router = _param(experts, h, std=h ** -0.5, **kw)
        self.w1 = _param(experts, hidden, h, std=h ** -0.5, **kw)
        self.w2 = _param(experts, h, hidden, std=hidden ** -0.5, **kw)
        self.register_buffer("bias", torch.zeros((experts,), dtype=torch.float32, device=device) if balance else None)

    def choose(self, y: torch.Tensor):
        """Each token's experts (int32) and their weights, of its normed rows y."""
        score = LinearActFunction.apply(y, self.router, None, None, MC2_ACT_NONE, None)
        if self.kind is not None:
            return RouteFunction.apply(score, self.bias, self.top, self.kind)
        top, ids = score.float().topk(self.top, dim=-1)
        return ids.to(torch.int32), torch.softmax(top, dim=-1)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        y, s = AddRMSNormFunction.apply(x, residual, self.norm, self.eps)
        ids, weights = self.choose(y)
        rows, row_map, offsets = PermuteFunction.apply(y, ids, self.experts)
        if self.keep8 and torch.is_grad_enabled():
            e = KeptLinearsFunction.apply(rows, self.w1, None, self.w2, None, None, self.act, offsets)
        else:
            a = LinearActFunction.apply(rows, self.w1, None, None, self.act, offsets)
            e = LinearActFunction.apply(a, self.w2, None, None, MC2_ACT_NONE, offsets)
        return UnpermuteFunction.apply(e, row_map, weights), s


class _Int8Linears(torch.nn.Module):
    """The two linears of a block as int8 codes with a scale per output channel."""

    def __init__(self, block):
        super().__init__()
        self.act, self.eps = block.act, block.eps
        for name in ("w1", "w2"):
            codes, scale = mc2_quant_rows(getattr(block, name).detach())
            self.register_buffer(name, codes)
            self.register_buffer(name + "_scale", scale)
        for name in ("norm", "b1", "b2"):
            value = getattr(block, name, None)
            self.register_buffer(name, None if value is None else value.detach().clone())

    def linears(self, q, scale, residual, group_offsets=None):
        a = mc2_linear_i8(q, scale, self.w1, self.w1_scale, self.b1, dtype=self.norm.dtype, act=self.act,
                          group_offsets=group_offsets)
        q, scale = mc2_quant_rows(a)
        return mc2_linear_i8(q, scale, self.w2, self.w2_scale, self.b2, residual, dtype=self.norm.dtype,
                             group_offsets=group_offsets)


class Int8FeedForward(_Int8Linears):
    """A FeedForward served in int8: the norm gives the codes that the first product reads."""

    @torch.no_grad()
    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        q, scale, s, _ = mc2_add_rms_norm(x, self.norm, residual, eps=self.eps, out_dtype=torch.int8)
        return self.linears(q, scale, s)


class Int8ExpertsFeedForward(_Int8Linears):
    """An ExpertsFeedForward served in int8: its router stays in 16 bits, and its choice the same."""

    def __init__(self, block: ExpertsFeedForward):
        super().__init__(block)
        self.experts, self.top, self.kind = block.experts, block.top, block.kind
        self.register_buffer("router", block.router.detach().clone())
        self.register_buffer("bias", None if block.bias is None else block.bias.clone())

    choose = ExpertsFeedForward.choose

    @torch.no_grad()
    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        y, _, s, _ = mc2_add_rms_norm(x, self.norm, residual, eps=self.eps)
        ids, weights = self.choose(y)
        rows, row_map, offsets = mc2_moe_permute(y, ids, self.experts)
        return mc2_moe_unpermute(self.linears(*mc2_quant_rows(rows), None, offsets), row_map, weights), s
