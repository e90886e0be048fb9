"""Binding of include/mc2_layer.h: the feed-forward operators around the MC2 matmuls.

``mc2_add_rms_norm``, ``mc2_linear_act``, ``mc2_moe_permute`` and
``mc2_moe_unpermute`` with their gradients, under the C names.  Like the rest
of the binding this only checks and marshals arguments; the work runs in
libmc2's HIP kernels.  Outputs and workspaces that are not given are allocated
on the stream the kernels run on; with a ``stream`` other than the current one
the inputs are recorded on it, so that their memory is not reused before the
kernels have read it.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import (_I64, _INT, _P, _TORCH_DT, _check, _lib, _stream_obj)

MC2_ACT_NONE, MC2_ACT_RELU, MC2_ACT_GELU, MC2_ACT_GELU_TANH, MC2_ACT_SILU = range(5)

_SZ, _FLT = ctypes.c_size_t, ctypes.c_float
_SZP = ctypes.POINTER(ctypes.c_size_t)
_SIGS = {
    "mc2_add_rms_norm": [_P, _P, _P, _I64, _I64, _INT, _FLT, _P, _INT, _P, _I64, _P, _P, _P],
    "mc2_add_rms_norm_grad_workspace_size": [_I64, _I64, _SZP],
    "mc2_add_rms_norm_grad": [_P, _P, _P, _P, _P, _I64, _I64, _INT, _P, _P, _P, _SZ, _P],
    "mc2_linear_act_workspace_size": [_I64, _I64, _I64, _I64, _SZP],
    "mc2_linear_act": [_P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _INT, _INT, _P, _P, _P, _SZ, _P],
    "mc2_linear_act_grad_workspace_size": [_I64, _I64, _I64, _I64, _SZP],
    "mc2_linear_act_grad": [_P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _INT, _INT, _P, _P, _P, _P, _SZ, _P],
    "mc2_moe_permute_workspace_size": [_I64, _I64, _I64, _SZP],
    "mc2_moe_permute": [_P, _P, _I64, _I64, _I64, _I64, _INT, _P, _P, _P, _P, _SZ, _P],
    "mc2_moe_unpermute": [_P, _P, _P, _I64, _I64, _I64, _I64, _INT, _P, _P],
    "mc2_moe_unpermute_grad": [_P, _P, _P, _P, _I64, _I64, _I64, _I64, _INT, _P, _P, _P],
}
for _name, _args in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int

_HALF = (torch.float16, torch.bfloat16)
_EIGHT = (torch.int8, torch.float8_e4m3fn)
_F32, _I32 = torch.float32, torch.int32


def _tensor(t, name: str, dim: Optional[int] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got shape {tuple(t.shape)}")
    return t.shape


def _half(t, name: str):
    if t.dtype not in _HALF:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")


def _like(t, name: str, shape, dtype):
    """An argument's shape and dtype (the C ABI sees only pointers and sizes)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _needed(t, name: str, shape, dtype):
    if t is None:
        raise ValueError(f"{name} is required")
    if t is not None:
        _like(t, name, shape, dtype)


def _place(names: str, *tensors) -> int:
    """The current stream's handle, after checking that every tensor is contiguous and on the
    current device (a decoding step's calls take a few microseconds: the checks are one pass)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            _refuse(names, tensors)
    if dev < 0 or dev != _current_device():
        _refuse(names, tensors)
    return torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None else _raw_stream(dev)


def _refuse(names: str, tensors):
    named = [(name, t) for name, t in zip(names.split(), tensors) if t is not None]
    for name, t in named:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    dev = None
    for name, t in named:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
        dev = t.device
    raise ValueError(f"tensors are on {dev} but the current device is cuda:{torch.cuda.current_device()}")


# the handle alone, without the Stream object around it, and the device without the check for a
# first use (a tensor on it is at hand)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(stream, fn, *args, **kwargs):
    """fn on another stream: its tensors are recorded there, and what it allocates is allocated there."""
    st = _stream_obj(stream)
    if st.cuda_stream != torch.cuda.current_stream().cuda_stream:
        for t in (*args, *kwargs.values()):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(st)
    with torch.cuda.stream(st):
        return fn(*args, **kwargs)


def _workspace(given, like, size_fn, *sizes):
    """(tensor, pointer, bytes) of a call's workspace; nothing where it needs none."""
    if given is not None:
        return given, given.data_ptr(), given.numel() * given.element_size()
    n = ctypes.c_size_t(0)
    _check(size_fn(*sizes, ctypes.byref(n)))
    if n.value == 0:
        return None, None, 0
    t = like.new_empty((n.value,), dtype=torch.uint8)
    return t, t.data_ptr(), n.value


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace_ok(t):
    if t is not None and (not isinstance(t, torch.Tensor) or t.dim() != 1):
        raise ValueError("workspace must be a 1-D tensor")


# ------------------------------------------------------------------ norm
def mc2_add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                     eps: float = 1e-6, out_dtype: Optional[torch.dtype] = None, group: int = 0,
                     need_rstd: bool = False, out: Optional[torch.Tensor] = None,
                     scale_out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                     rstd_out: Optional[torch.Tensor] = None, stream=None
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """s = x + residual, out = s / sqrt(mean(s^2) + eps) * weight over x's last dimension.

    Returns (out, scale, sum, rstd).  out_dtype torch.int8 or torch.float8_e4m3fn gives codes
    with fp32 scales per row (group 0, scale (rows, 1)) or per 128 columns (group 128); scale is
    None for the 16-bit output.  sum is s in x's dtype: x itself without a residual.  rstd (rows)
    fp32 comes with need_rstd, for mc2_add_rms_norm_grad.
    """
    if stream is not None:
        return _on(stream, mc2_add_rms_norm, x, weight, residual, eps=eps, out_dtype=out_dtype, group=group,
                   need_rstd=need_rstd, out=out, scale_out=scale_out, sum_out=sum_out, rstd_out=rstd_out)
    shape = _tensor(x, "x")
    if len(shape) < 1:
        raise ValueError("x must have a last dimension")
    h = shape[-1]
    rows = x.numel() // h if h else 0
    _half(x, "x")
    dt = x.dtype
    if out is not None:
        _tensor(out, "out")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = dt
    eight = out_dtype in _EIGHT
    if not eight and out_dtype != dt:
        raise TypeError(f"out_dtype must be {dt}, int8 or float8_e4m3fn, got {out_dtype}")
    if group not in (0, 128) or (group and (not eight or h % 128)):
        raise ValueError("group must be 0, or 128 with an 8-bit output and a multiple of 128 columns")
    scales = (rows, h // group if group else 1)
    _needed(weight, "weight", (h,), dt)
    if residual is not None:
        _like(residual, "residual", shape, dt)
    if out is not None:
        _like(out, "out", shape, out_dtype)
    if sum_out is not None:
        _like(sum_out, "sum_out", shape, dt)
    if rstd_out is not None:
        _like(rstd_out, "rstd_out", (rows,), _F32)
    if scale_out is not None:
        if not eight:
            raise ValueError("scale_out goes with an 8-bit output")
        _like(scale_out, "scale_out", scales, _F32)
    handle = _place("x weight residual out scale_out sum_out rstd_out", x, weight, residual, out, scale_out, sum_out,
                    rstd_out)
    if out is None:
        out = torch.empty_like(x) if not eight else x.new_empty(shape, dtype=out_dtype)
    if eight and scale_out is None:
        scale_out = x.new_empty(scales, dtype=_F32)
    if residual is not None and sum_out is None:
        sum_out = torch.empty_like(x)
    if need_rstd and rstd_out is None:
        rstd_out = x.new_empty((rows,), dtype=_F32)
    _check(_lib.mc2_add_rms_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), rows, h, _TORCH_DT[dt], eps,
                                 out.data_ptr(), _TORCH_DT[out_dtype], _ptr(scale_out), group, _ptr(sum_out),
                                 _ptr(rstd_out), handle))
    return out, scale_out, x if sum_out is None else sum_out, rstd_out


def mc2_add_rms_norm_grad(dout: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          dsum: Optional[torch.Tensor] = None, *, dx: Optional[torch.Tensor] = None,
                          dweight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight) of mc2_add_rms_norm's 16-bit output; s and rstd are its sum and rstd, dsum the
    gradient that reached sum.  dx is the gradient of x and of residual."""
    if stream is not None:
        return _on(stream, mc2_add_rms_norm_grad, dout, s, weight, rstd, dsum, dx=dx, dweight=dweight,
                   workspace=workspace)
    shape = _tensor(s, "s")
    if len(shape) < 1:
        raise ValueError("s must have a last dimension")
    h = shape[-1]
    rows = s.numel() // h if h else 0
    _half(s, "s")
    dt = s.dtype
    _needed(dout, "dout", shape, dt)
    _needed(weight, "weight", (h,), dt)
    _needed(rstd, "rstd", (rows,), _F32)
    if dsum is not None:
        _like(dsum, "dsum", shape, dt)
    if dx is not None:
        _like(dx, "dx", shape, dt)
    if dweight is not None:
        _like(dweight, "dweight", (h,), dt)
    _workspace_ok(workspace)
    handle = _place("dout s weight rstd dsum dx dweight workspace", dout, s, weight, rstd, dsum, dx, dweight, workspace)
    _ws, ws, ws_bytes = _workspace(workspace, s, _lib.mc2_add_rms_norm_grad_workspace_size, rows, h)
    if dx is None:
        dx = torch.empty_like(s)
    if dweight is None:
        dweight = torch.empty_like(weight)
    _check(_lib.mc2_add_rms_norm_grad(dout.data_ptr(), _ptr(dsum), s.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                                      rows, h, _TORCH_DT[dt], dx.data_ptr(), dweight.data_ptr(), ws, ws_bytes, handle))
    return dx, dweight


# ------------------------------------------------------------------ linear
def _linear_sizes(x, w, group_offsets, half: bool = True, w_dtype: Optional[torch.dtype] = None):
    m, k = _tensor(x, "x", 2)
    if half:
        _half(x, "x")
    groups = 0
    if group_offsets is not None:
        (size,) = _tensor(group_offsets, "group_offsets", 1)
        groups = size - 1
        if groups < 1:
            raise ValueError("group_offsets must hold at least 2 values")
        if group_offsets.dtype != _I32:
            raise TypeError(f"group_offsets has dtype {group_offsets.dtype}, expected torch.int32")
    n = _tensor(w, "w", 3 if groups else 2)[-2]
    _needed(w, "w", (groups, n, k) if groups else (n, k), w_dtype or x.dtype)
    return m, k, n, groups


def mc2_linear_act(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, *, act: int = MC2_ACT_NONE,
                   group_offsets: Optional[torch.Tensor] = None, need_z: bool = False,
                   out: Optional[torch.Tensor] = None, z_out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """out = residual + act(x @ w^T + bias): returns (out, z), z the pre-activation with need_z.

    x (m, k), w (n, k) in the nn.Linear layout, bias (n), residual (m, n).  With group_offsets
    (G + 1 int32 on the device) w is (G, n, k), bias (G, n), and rows group_offsets[g] ..
    group_offsets[g + 1] use matrix g; rows after the last range get z = 0.
    """
    if stream is not None:
        return _on(stream, mc2_linear_act, x, w, bias, residual, act=act, group_offsets=group_offsets, need_z=need_z,
                   out=out, z_out=z_out, workspace=workspace)
    m, k, n, groups = _linear_sizes(x, w, group_offsets)
    dt = x.dtype
    if bias is not None:
        _like(bias, "bias", (groups, n) if groups else (n,), dt)
    if residual is not None:
        _like(residual, "residual", (m, n), dt)
    if out is not None:
        _like(out, "out", (m, n), dt)
    if z_out is not None:
        _like(z_out, "z_out", (m, n), dt)
    _workspace_ok(workspace)
    handle = _place("x w bias residual group_offsets out z_out workspace", x, w, bias, residual, group_offsets, out,
                    z_out, workspace)
    _ws, ws, ws_bytes = _workspace(workspace, x, _lib.mc2_linear_act_workspace_size, m, k, n, groups)
    if out is None:
        out = x.new_empty((m, n))
    if need_z and z_out is None:
        z_out = x.new_empty((m, n))
    _check(_lib.mc2_linear_act(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), m, k, n, _ptr(group_offsets),
                               groups, _TORCH_DT[dt], act, out.data_ptr(), _ptr(z_out), ws, ws_bytes, handle))
    return out, z_out


def mc2_linear_act_grad(dout: torch.Tensor, x: torch.Tensor, w: torch.Tensor, z: Optional[torch.Tensor] = None, *,
                        act: int = MC2_ACT_NONE, group_offsets: Optional[torch.Tensor] = None, need_dx: bool = True,
                        need_dw: bool = True, need_dbias: bool = False, dx: Optional[torch.Tensor] = None,
                        dw: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dw, dbias) of mc2_linear_act, each None unless wanted (need_*, or given); z is its
    pre-activation (not needed with MC2_ACT_NONE).  The residual's gradient is dout itself."""
    if stream is not None:
        return _on(stream, mc2_linear_act_grad, dout, x, w, z, act=act, group_offsets=group_offsets, need_dx=need_dx,
                   need_dw=need_dw, need_dbias=need_dbias, dx=dx, dw=dw, dbias=dbias, workspace=workspace)
    m, k, n, groups = _linear_sizes(x, w, group_offsets)
    dt = x.dtype
    bias_shape = (groups, n) if groups else (n,)
    _needed(dout, "dout", (m, n), dt)
    if act != MC2_ACT_NONE:
        _needed(z, "z", (m, n), dt)
    elif z is not None:
        _like(z, "z", (m, n), dt)
    if dx is not None:
        _like(dx, "dx", (m, k), dt)
    if dw is not None:
        _like(dw, "dw", w.shape, dt)
    if dbias is not None:
        _like(dbias, "dbias", bias_shape, dt)
    _workspace_ok(workspace)
    handle = _place("dout x w z group_offsets dx dw dbias workspace", dout, x, w, z, group_offsets, dx, dw, dbias,
                    workspace)
    _ws, ws, ws_bytes = _workspace(workspace, x, _lib.mc2_linear_act_grad_workspace_size, m, k, n, groups)
    if need_dx and dx is None:
        dx = torch.empty_like(x)
    if need_dw and dw is None:
        dw = torch.empty_like(w)
    if need_dbias and dbias is None:
        dbias = x.new_empty(bias_shape)
    _check(_lib.mc2_linear_act_grad(dout.data_ptr(), _ptr(z), x.data_ptr(), w.data_ptr(), m, k, n, _ptr(group_offsets),
                                    groups, _TORCH_DT[dt], act, _ptr(dx), _ptr(dw), _ptr(dbias), ws, ws_bytes, handle))
    return dx, dw, dbias


# ------------------------------------------------------------------ tokens by expert
def mc2_moe_permute(x: torch.Tensor, expert_ids: torch.Tensor, experts: int, *, out: Optional[torch.Tensor] = None,
                    row_map: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Rows of x (tokens, h) for every choice expert_ids[t][j] (int32), sorted by expert and then by
    t * top + j: returns (out (tokens * top, h), row_map (tokens, top) int32, offsets (experts + 1)
    int32).  Ids outside [0, experts) are dropped: row_map -1; out's last rows are then 0."""
    if stream is not None:
        return _on(stream, mc2_moe_permute, x, expert_ids, experts, out=out, row_map=row_map, offsets=offsets,
                   workspace=workspace)
    tokens, h = _tensor(x, "x", 2)
    _half(x, "x")
    top = _tensor(expert_ids, "expert_ids", 2)[1]
    _needed(expert_ids, "expert_ids", (tokens, top), _I32)
    if out is not None:
        _like(out, "out", (tokens * top, h), x.dtype)
    if row_map is not None:
        _like(row_map, "row_map", (tokens, top), _I32)
    if offsets is not None:
        _like(offsets, "offsets", (experts + 1,), _I32)
    _workspace_ok(workspace)
    handle = _place("x expert_ids out row_map offsets workspace", x, expert_ids, out, row_map, offsets, workspace)
    _ws, ws, ws_bytes = _workspace(workspace, x, _lib.mc2_moe_permute_workspace_size, tokens, top, experts)
    if out is None:
        out = x.new_empty((tokens * top, h))
    if row_map is None:
        row_map = torch.empty_like(expert_ids)
    if offsets is None:
        offsets = expert_ids.new_empty((experts + 1,))
    _check(_lib.mc2_moe_permute(x.data_ptr(), expert_ids.data_ptr(), tokens, top, h, experts, _TORCH_DT[x.dtype],
                                out.data_ptr(), row_map.data_ptr(), offsets.data_ptr(), ws, ws_bytes, handle))
    return out, row_map, offsets


def mc2_moe_unpermute(y: torch.Tensor, row_map: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum over j of weights[t][j] * y[row_map[t][j]] (weights (tokens, top) fp32, or None
    for 1).  Without weights it is also mc2_moe_permute's gradient."""
    if stream is not None:
        return _on(stream, mc2_moe_unpermute, y, row_map, weights, out=out)
    rows, h = _tensor(y, "y", 2)
    _half(y, "y")
    tokens, top = _tensor(row_map, "row_map", 2)
    _needed(row_map, "row_map", (tokens, top), _I32)
    if weights is not None:
        _like(weights, "weights", (tokens, top), _F32)
    if out is not None:
        _like(out, "out", (tokens, h), y.dtype)
    handle = _place("y row_map weights out", y, row_map, weights, out)
    if out is None:
        out = y.new_empty((tokens, h))
    _check(_lib.mc2_moe_unpermute(y.data_ptr(), row_map.data_ptr(), _ptr(weights), tokens, top, h, rows,
                                  _TORCH_DT[y.dtype], out.data_ptr(), handle))
    return out


def mc2_moe_unpermute_grad(dout: torch.Tensor, y: torch.Tensor, row_map: torch.Tensor,
                           weights: Optional[torch.Tensor] = None, *, need_dweights: bool = True,
                           dy: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None, stream=None
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(dy, dweights) of mc2_moe_unpermute for a row_map that mc2_moe_permute gave."""
    if stream is not None:
        return _on(stream, mc2_moe_unpermute_grad, dout, y, row_map, weights, need_dweights=need_dweights, dy=dy,
                   dweights=dweights)
    rows, h = _tensor(y, "y", 2)
    _half(y, "y")
    tokens, top = _tensor(row_map, "row_map", 2)
    _needed(row_map, "row_map", (tokens, top), _I32)
    _needed(dout, "dout", (tokens, h), y.dtype)
    if weights is not None:
        _like(weights, "weights", (tokens, top), _F32)
    if dy is not None:
        _like(dy, "dy", (rows, h), y.dtype)
    if dweights is not None:
        _like(dweights, "dweights", (tokens, top), _F32)
    handle = _place("dout y row_map weights dy dweights", dout, y, row_map, weights, dy, dweights)
    if dy is None:
        dy = torch.empty_like(y)
    if need_dweights and dweights is None:
        dweights = y.new_empty((tokens, top), dtype=_F32)
    _check(_lib.mc2_moe_unpermute_grad(dout.data_ptr(), y.data_ptr(), row_map.data_ptr(), _ptr(weights), tokens, top,
                                       h, rows, _TORCH_DT[y.dtype], dy.data_ptr(), _ptr(dweights), handle))
    return dy, dweights


__all__ = ["MC2_ACT_NONE", "MC2_ACT_RELU", "MC2_ACT_GELU", "MC2_ACT_GELU_TANH", "MC2_ACT_SILU",
           "mc2_add_rms_norm", "mc2_add_rms_norm_grad", "mc2_linear_act", "mc2_linear_act_grad", "mc2_moe_permute",
           "mc2_moe_unpermute", "mc2_moe_unpermute_grad"]
