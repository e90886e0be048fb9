"""Binding of include/mc2_layer8.h: the router, and the feed-forward operators' 8-bit forms.

``mc2_moe_route`` and its gradient, ``mc2_quant_rows`` / ``mc2_dequant_rows``,
``mc2_linear_i8``, and ``mc2_linear_act_grad_i8``, under the C names.  As in
layer.py this only checks and marshals arguments, outputs and workspaces that
are not given are allocated on the stream the kernels run on, and with a
``stream`` other than the current one the inputs are recorded on it.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _I64, _INT, _P, _TORCH_DT, _check, _lib
from .layer import (_F32, _FLT, _HALF, _I32, _SZ, _SZP, MC2_ACT_NONE, _half, _like, _linear_sizes, _needed, _on, _place,
                    _ptr, _tensor, _workspace_ok)

MC2_SCORE_SOFTMAX, MC2_SCORE_SIGMOID = range(2)
MC2_SCORE_KEEP_NAN = MC2_KEEP_INF = 1 << 16

_SIGS = {
    "mc2_moe_route": [_P, _P, _I64, _I64, _I64, _INT, _INT, _I64, _I64, _I64, _INT, _FLT, _P, _P, _P],
    "mc2_moe_route_grad": [_P, _P, _P, _I64, _I64, _I64, _INT, _INT, _INT, _FLT, _P, _P],
    "mc2_quant_rows": [_P, _I64, _I64, _INT, _I64, _P, _P, _P],
    "mc2_dequant_rows": [_P, _P, _I64, _I64, _I64, _INT, _INT, _P, _P],
    "mc2_linear_i8_workspace_size": [_I64, _I64, _I64, _I64, _SZP],
    "mc2_linear_i8": [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _INT, _INT, _P, _P, _SZ, _P],
    "mc2_linear_act_grad_i8_workspace_size": [_I64, _I64, _I64, _I64, _SZP],
    "mc2_linear_act_grad_i8": [_P, _P, _P, _P, _P, _INT, _P, _I64, _I64, _I64, _P, _I64, _INT, _INT, _P, _P, _P, _P,
                               _SZ, _P],
}
for _name, _args in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int

_I8 = torch.int8
_LOGITS = (torch.float32,) + _HALF


@functools.lru_cache(maxsize=4096)
def _bytes(size_fn: str, m: int, k: int, n: int, groups: int) -> int:
    """A workspace's size, which depends on these alone (asking the library takes longer than a decoding step's other
    checks together)."""
    size = ctypes.c_size_t(0)
    _check(getattr(_lib, size_fn)(m, k, n, groups, ctypes.byref(size)))
    return size.value


def _space(given, like, size_fn: str, *sizes):
    """(tensor, pointer, bytes) of a call's workspace; nothing where it needs none."""
    if given is not None:
        return given, given.data_ptr(), given.numel() * given.element_size()
    size = _bytes(size_fn, *sizes)
    if size == 0:
        return None, None, 0
    t = like.new_empty((size,), dtype=torch.uint8)
    return t, t.data_ptr(), size


def _codes(t, name: str):
    if t.dtype != _I8:
        raise TypeError(f"{name} must be int8, got {t.dtype}")


# ------------------------------------------------------------------ router
def mc2_moe_route(logits: torch.Tensor, top: int, bias: Optional[torch.Tensor] = None, *,
                  score: int = MC2_SCORE_SOFTMAX, groups: int = 1, top_groups: int = 1, group_top: int = 1,
                  renormalise: bool = True, scale: float = 1.0, keep_nan: bool = False,
                  expert_ids: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None, stream=None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(expert_ids (tokens, top) int32, weights (tokens, top) fp32) of logits (tokens, experts), fp32 or 16-bit.

    The `top` experts of the largest score + bias, in descending order (equal ones: the lowest first; without a bias by
    their logits, also where the scores round to equal numbers); the weights are their scores (without the bias)
    times scale, with renormalise over their sum.  groups > 1: only experts of the top_groups groups of neighbours
    whose group_top (1 or 2) largest sum to most.  A logit of -inf turns an expert off; an id is -1 (weight 0) where
    too few are on, and all are (weights NaN) for a token with a NaN, or under a softmax a logit of +inf.  With keep_nan
    such a token has the experts 0 .. top - 1, through which its weights make its row of mc2_moe_unpermute NaN.
    """
    if stream is not None:
        return _on(stream, mc2_moe_route, logits, top, bias, score=score, groups=groups, top_groups=top_groups,
                   group_top=group_top, renormalise=renormalise, scale=scale, keep_nan=keep_nan, expert_ids=expert_ids,
                   weights=weights)
    tokens, experts = _tensor(logits, "logits", 2)
    if logits.dtype not in _LOGITS:
        raise TypeError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
    if bias is not None:
        _like(bias, "bias", (experts,), _F32)
    if expert_ids is not None:
        _like(expert_ids, "expert_ids", (tokens, top), _I32)
    if weights is not None:
        _like(weights, "weights", (tokens, top), _F32)
    handle = _place("logits bias expert_ids weights", logits, bias, expert_ids, weights)
    if top < 1 or top > experts:
        raise ValueError(f"top must lie in [1, experts], got {top}")
    if expert_ids is None:
        expert_ids = logits.new_empty((tokens, top), dtype=_I32)
    if weights is None:
        weights = logits.new_empty((tokens, top), dtype=_F32)
    _check(_lib.mc2_moe_route(logits.data_ptr(), _ptr(bias), tokens, experts, top, _TORCH_DT[logits.dtype],
                              score + MC2_SCORE_KEEP_NAN if keep_nan else score, groups, top_groups, group_top,
                              bool(renormalise), scale, expert_ids.data_ptr(), weights.data_ptr(), handle))
    return expert_ids, weights


def mc2_moe_route_grad(dweights: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor, *,
                       score: int = MC2_SCORE_SOFTMAX, renormalise: bool = True, scale: float = 1.0,
                       dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of mc2_moe_route's weights for its logits, at the experts it chose.  Ids outside the experts have
    no part in it.  dlogits may be logits itself."""
    if stream is not None:
        return _on(stream, mc2_moe_route_grad, dweights, logits, expert_ids, score=score, renormalise=renormalise,
                   scale=scale, dlogits=dlogits)
    tokens, experts = _tensor(logits, "logits", 2)
    if logits.dtype not in _LOGITS:
        raise TypeError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
    top = _tensor(expert_ids, "expert_ids", 2)[1]
    _like(expert_ids, "expert_ids", (tokens, top), _I32)
    _needed(dweights, "dweights", (tokens, top), _F32)
    if dlogits is not None:
        _like(dlogits, "dlogits", (tokens, experts), logits.dtype)
    handle = _place("dweights logits expert_ids dlogits", dweights, logits, expert_ids, dlogits)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    _check(_lib.mc2_moe_route_grad(dweights.data_ptr(), logits.data_ptr(), expert_ids.data_ptr(), tokens, experts, top,
                                   _TORCH_DT[logits.dtype], score, bool(renormalise), scale, dlogits.data_ptr(), handle))
    return dlogits


# ------------------------------------------------------------------ int8 codes of rows
def _scales(cols: int, group: int) -> int:
    return -(-cols // 128) if group else 1


def mc2_quant_rows(x: torch.Tensor, *, group: int = 0, keep_inf: bool = False, codes: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(int8 codes of x's shape, fp32 scale): max |x| / 127 per row of x's last dimension (group 0, scale (..., 1)) or
    per 128 of its columns (group 128, scale (..., ceil(columns / 128))), and rint(x / scale).

    A group with an infinity or a NaN comes back as NaN.  With keep_inf (group 128; for pre-activations) infinities
    do not count for the scale: +inf becomes the largest finite value of its group, and -inf stays one."""
    if stream is not None:
        return _on(stream, mc2_quant_rows, x, group=group, keep_inf=keep_inf, codes=codes, scale=scale)
    shape = _tensor(x, "x")
    if len(shape) < 1:
        raise ValueError("x must have a last dimension")
    _half(x, "x")
    if group not in (0, 128):
        raise ValueError(f"group must be 0 or 128, got {group}")
    if keep_inf and group != 128:
        raise ValueError("keep_inf needs group 128")
    cols = shape[-1]
    scales = (*shape[:-1], _scales(cols, group))
    if codes is not None:
        _like(codes, "codes", shape, _I8)
    if scale is not None:
        _like(scale, "scale", scales, _F32)
    handle = _place("x codes scale", x, codes, scale)
    if codes is None:
        codes = x.new_empty(shape, dtype=_I8)
    if scale is None:
        scale = x.new_empty(scales, dtype=_F32)
    _check(_lib.mc2_quant_rows(x.data_ptr(), x.numel() // cols if cols else 0, cols, _TORCH_DT[x.dtype],
                               group + MC2_KEEP_INF if keep_inf else group, codes.data_ptr(), scale.data_ptr(), handle))
    return codes, scale


def mc2_dequant_rows(codes: torch.Tensor, scale: torch.Tensor, *, group: int = 0, act: int = MC2_ACT_NONE,
                     dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None
                     ) -> torch.Tensor:
    """act(codes * scale) in dtype (that of out, where given): mc2_quant_rows' values, through an activation."""
    if stream is not None:
        return _on(stream, mc2_dequant_rows, codes, scale, group=group, act=act, dtype=dtype, out=out)
    shape = _tensor(codes, "codes")
    if len(shape) < 1:
        raise ValueError("codes must have a last dimension")
    _codes(codes, "codes")
    if group not in (0, 128):
        raise ValueError(f"group must be 0 or 128, got {group}")
    cols = shape[-1]
    _needed(scale, "scale", (*shape[:-1], _scales(cols, group)), _F32)
    if out is not None:
        _tensor(out, "out")
        dtype = out.dtype
    if dtype not in _HALF:
        raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
    if out is not None:
        _like(out, "out", shape, dtype)
    handle = _place("codes scale out", codes, scale, out)
    if out is None:
        out = codes.new_empty(shape, dtype=dtype)
    _check(_lib.mc2_dequant_rows(codes.data_ptr(), scale.data_ptr(), codes.numel() // cols if cols else 0, cols, group,
                                 act, _TORCH_DT[dtype], out.data_ptr(), handle))
    return out


# ------------------------------------------------------------------ linear of int8 codes
def _scale_of_rows(t, name: str, rows):
    """fp32 scales of a shape, or of it with a last dimension of 1, as mc2_quant_rows gives them."""
    if t is None:
        raise ValueError(f"{name} is required")
    if isinstance(t, torch.Tensor) and t.dim() == len(rows) + 1:
        _like(t, name, (*rows, 1), _F32)
    else:
        _like(t, name, rows, _F32)


def mc2_linear_i8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                  bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, *,
                  dtype: Optional[torch.dtype] = None, act: int = MC2_ACT_NONE,
                  group_offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out = residual + act((x @ w^T) * x_scale * w_scale + bias) of int8 codes x (m, k) and w (n, k).

    x_scale (m) or (m, 1) and w_scale (n) or (n, 1), fp32: one scale for each token and channel, as mc2_quant_rows
    and mc2_add_rms_norm give them.  bias (n), residual and out (m, n) are of dtype: float16 or bfloat16, that of
    whichever is given, else bfloat16.  group_offsets as in mc2_linear_act: then w is (G, n, k), w_scale (G, n) or
    (G, n, 1), bias (G, n).
    """
    if stream is not None:
        return _on(stream, mc2_linear_i8, x, x_scale, w, w_scale, bias, residual, dtype=dtype, act=act,
                   group_offsets=group_offsets, out=out, workspace=workspace)
    _tensor(x, "x", 2)
    _codes(x, "x")
    m, k, n, groups = _linear_sizes(x, w, group_offsets, half=False)
    channels = (groups, n) if groups else (n,)
    _scale_of_rows(x_scale, "x_scale", (m,))
    _scale_of_rows(w_scale, "w_scale", channels)
    for t in (out, residual, bias):
        if dtype is None and isinstance(t, torch.Tensor):
            dtype = t.dtype
    if dtype is None:
        dtype = torch.bfloat16
    if dtype not in _HALF:
        raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
    if bias is not None:
        _like(bias, "bias", channels, dtype)
    if residual is not None:
        _like(residual, "residual", (m, n), dtype)
    if out is not None:
        _like(out, "out", (m, n), dtype)
    _workspace_ok(workspace)
    handle = _place("x x_scale w w_scale bias residual group_offsets out workspace", x, x_scale, w, w_scale, bias,
                    residual, group_offsets, out, workspace)
    _ws, ws, ws_bytes = _space(workspace, x, "mc2_linear_i8_workspace_size", m, k, n, groups)
    if out is None:
        out = x.new_empty((m, n), dtype=dtype)
    _check(_lib.mc2_linear_i8(x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), _ptr(bias),
                              _ptr(residual), m, k, n, _ptr(group_offsets), groups, _TORCH_DT[dtype], act,
                              out.data_ptr(), ws, ws_bytes, handle))
    return out


# ------------------------------------------------------------------ gradients from what was kept in 8 bits
def mc2_linear_act_grad_i8(dout: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor,
                           z: Optional[torch.Tensor] = None, z_scale: Optional[torch.Tensor] = None, *,
                           act: int = MC2_ACT_NONE, x_act: int = MC2_ACT_NONE,
                           group_offsets: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True,
                           need_dbias: bool = False, dx: Optional[torch.Tensor] = None,
                           dw: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None
                           ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dw, dbias) of mc2_linear_act from int8 codes of its input and its pre-activation.

    x (m, k) and z (m, n) int8 with x_scale (m, ceil(k / 128)) and z_scale (m, ceil(n / 128)), as mc2_quant_rows
    gives them with group 128; the linear's input was x_act(x * x_scale).  z is not needed with MC2_ACT_NONE.
    dout (m, n) and w are 16-bit, and so are the gradients; each is None unless wanted (need_*, or given).
    """
    if stream is not None:
        return _on(stream, mc2_linear_act_grad_i8, dout, x, x_scale, w, z, z_scale, act=act, x_act=x_act,
                   group_offsets=group_offsets, need_dx=need_dx, need_dw=need_dw, need_dbias=need_dbias, dx=dx, dw=dw,
                   dbias=dbias, workspace=workspace)
    _tensor(x, "x", 2)
    _codes(x, "x")
    _tensor(w, "w")
    _half(w, "w")
    dt = w.dtype
    m, k, n, groups = _linear_sizes(x, w, group_offsets, half=False, w_dtype=dt)
    bias_shape = (groups, n) if groups else (n,)
    _needed(dout, "dout", (m, n), dt)
    _needed(x_scale, "x_scale", (m, _scales(k, 128)), _F32)
    if act != MC2_ACT_NONE:
        _needed(z, "z", (m, n), _I8)
        _needed(z_scale, "z_scale", (m, _scales(n, 128)), _F32)
    else:
        if z is not None:
            _like(z, "z", (m, n), _I8)
        if z_scale is not None:
            _like(z_scale, "z_scale", (m, _scales(n, 128)), _F32)
    if dx is not None:
        _like(dx, "dx", (m, k), dt)
    if dw is not None:
        _like(dw, "dw", w.shape, dt)
    if dbias is not None:
        _like(dbias, "dbias", bias_shape, dt)
    _workspace_ok(workspace)
    handle = _place("dout x x_scale w z z_scale group_offsets dx dw dbias workspace", dout, x, x_scale, w, z, z_scale,
                    group_offsets, dx, dw, dbias, workspace)
    _ws, ws, ws_bytes = _space(workspace, x, "mc2_linear_act_grad_i8_workspace_size", m, k, n, groups)
    if need_dx and dx is None:
        dx = dout.new_empty((m, k))
    if need_dw and dw is None:
        dw = torch.empty_like(w)
    if need_dbias and dbias is None:
        dbias = dout.new_empty(bias_shape)
    _check(_lib.mc2_linear_act_grad_i8(dout.data_ptr(), _ptr(z), _ptr(z_scale), x.data_ptr(), x_scale.data_ptr(), x_act,
                                       w.data_ptr(), m, k, n, _ptr(group_offsets), groups, _TORCH_DT[dt], act, _ptr(dx),
                                       _ptr(dw), _ptr(dbias), ws, ws_bytes, handle))
    return dx, dw, dbias


__all__ = ["MC2_SCORE_SOFTMAX", "MC2_SCORE_SIGMOID", "MC2_SCORE_KEEP_NAN", "MC2_KEEP_INF", "mc2_moe_route",
           "mc2_moe_route_grad", "mc2_quant_rows", "mc2_dequant_rows", "mc2_linear_i8", "mc2_linear_act_grad_i8"]
