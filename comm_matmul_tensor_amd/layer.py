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

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import (_I64, _INT, _P, _TORCH_DT, _check, _lib, _stream_obj)

MC2_ACT_NONE, MC2_ACT_RELU, MC2_ACT_GELU, MC2_ACT_GELU_TANH, MC2_ACT_SILU = range(5)

_SZ, _F32 = ctypes.c_size_t, ctypes.c_float
_SZP = ctypes.POINTER(ctypes.c_size_t)
_SIGS = {
    "mc2_add_rms_norm": [_P, _P, _P, _I64, _I64, _INT, _F32, _P, _INT, _P, _I64, _P, _P, _P],
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
    """An optional argument's shape and dtype (the C ABI sees only pointers and sizes)."""
    if t is None:
        return
    _tensor(t, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _needed(t, name: str, shape, dtype):
    if t is None:
        raise ValueError(f"{name} is required")
    _like(t, name, shape, dtype)


class _Call:
    """Where a call runs: the tensors' device, which must be the current one, and the stream."""

    def __init__(self, stream, **named):
        dev = None
        for name, t in named.items():
            if t is None:
                continue
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if not t.is_cuda:
                raise ValueError(f"{name} must be a device tensor")
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
        current = torch.cuda.current_device()
        if dev.index != current:
            raise ValueError(f"tensors are on {dev} but the current device is cuda:{current}")
        self.device = dev
        now = torch.cuda.current_stream()
        if stream is None:
            self.handle, self.scope = now.cuda_stream, contextlib.nullcontext()
            return
        st = _stream_obj(stream)
        self.handle, self.scope = st.cuda_stream, torch.cuda.stream(st)
        if st.cuda_stream != now.cuda_stream:
            for t in named.values():
                if t is not None:
                    t.record_stream(st)

    def empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, given, size_fn: str, *sizes):
        """The workspace tensor of a call (None where it needs none)."""
        n = ctypes.c_size_t(0)
        _check(getattr(_lib, size_fn)(*sizes, ctypes.byref(n)))
        if given is not None:
            return given
        return self.empty((n.value,), torch.uint8) if n.value else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


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
    shape = _tensor(x, "x")
    if len(shape) < 1:
        raise ValueError("x must have a last dimension")
    h = shape[-1]
    rows = x.numel() // h if h else 0
    _half(x, "x")
    dt = x.dtype
    if out is not None:
        out_dtype = _tensor(out, "out") and out.dtype
    out_dtype = out_dtype or dt
    eight = out_dtype in (torch.int8, torch.float8_e4m3fn)
    if not eight and out_dtype != dt:
        raise TypeError(f"out_dtype must be {dt}, int8 or float8_e4m3fn, got {out_dtype}")
    if group not in (0, 128) or (group and (not eight or h % 128)):
        raise ValueError("group must be 0, or 128 with an 8-bit output and a multiple of 128 columns")
    scales = (rows, h // group if group else 1)
    _needed(weight, "weight", (h,), dt)
    _like(residual, "residual", shape, dt)
    _like(out, "out", shape, out_dtype)
    _like(sum_out, "sum_out", shape, dt)
    _like(rstd_out, "rstd_out", (rows,), torch.float32)
    if scale_out is not None and not eight:
        raise ValueError("scale_out goes with an 8-bit output")
    _like(scale_out, "scale_out", scales, torch.float32)
    call = _Call(stream, x=x, weight=weight, residual=residual, out=out, scale_out=scale_out, sum_out=sum_out,
                 rstd_out=rstd_out)
    with call.scope:
        if out is None:
            out = call.empty(shape, out_dtype)
        if eight and scale_out is None:
            scale_out = call.empty(scales, torch.float32)
        if residual is not None and sum_out is None:
            sum_out = call.empty(shape, dt)
        if need_rstd and rstd_out is None:
            rstd_out = call.empty((rows,), torch.float32)
        _check(_lib.mc2_add_rms_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), rows, h, _TORCH_DT[dt], eps,
                                     out.data_ptr(), _TORCH_DT[out_dtype], _ptr(scale_out), group, _ptr(sum_out),
                                     _ptr(rstd_out), call.handle))
    return out, scale_out, x if sum_out is None else sum_out, rstd_out


def mc2_add_rms_norm_grad(dout: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          dsum: Optional[torch.Tensor] = None, *, dx: Optional[torch.Tensor] = None,
                          dweight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight) of mc2_add_rms_norm's 16-bit output; s and rstd are its sum and rstd, dsum the
    gradient that reached sum.  dx is the gradient of x and of residual."""
    shape = _tensor(s, "s")
    if len(shape) < 1:
        raise ValueError("s must have a last dimension")
    h = shape[-1]
    rows = s.numel() // h if h else 0
    _half(s, "s")
    dt = s.dtype
    _needed(dout, "dout", shape, dt)
    _needed(weight, "weight", (h,), dt)
    _needed(rstd, "rstd", (rows,), torch.float32)
    _like(dsum, "dsum", shape, dt)
    _like(dx, "dx", shape, dt)
    _like(dweight, "dweight", (h,), dt)
    _workspace_ok(workspace)
    call = _Call(stream, dout=dout, s=s, weight=weight, rstd=rstd, dsum=dsum, dx=dx, dweight=dweight,
                 workspace=workspace)
    with call.scope:
        workspace = call.workspace(workspace, "mc2_add_rms_norm_grad_workspace_size", rows, h)
        if dx is None:
            dx = call.empty(shape, dt)
        if dweight is None:
            dweight = call.empty((h,), dt)
        _check(_lib.mc2_add_rms_norm_grad(dout.data_ptr(), _ptr(dsum), s.data_ptr(), weight.data_ptr(),
                                          rstd.data_ptr(), rows, h, _TORCH_DT[dt], dx.data_ptr(), dweight.data_ptr(),
                                          _ptr(workspace), _bytes(workspace), call.handle))
    return dx, dweight


# ------------------------------------------------------------------ linear
def _linear_sizes(x, w, group_offsets):
    m, k = _tensor(x, "x", 2)
    _half(x, "x")
    groups = 0
    if group_offsets is not None:
        (size,) = _tensor(group_offsets, "group_offsets", 1)
        groups = size - 1
        if groups < 1:
            raise ValueError("group_offsets must hold at least 2 values")
        if group_offsets.dtype != torch.int32:
            raise TypeError(f"group_offsets has dtype {group_offsets.dtype}, expected torch.int32")
    n = _tensor(w, "w", 3 if groups else 2)[-2]
    _needed(w, "w", (groups, n, k) if groups else (n, k), x.dtype)
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
    m, k, n, groups = _linear_sizes(x, w, group_offsets)
    dt = x.dtype
    _like(bias, "bias", (groups, n) if groups else (n,), dt)
    _like(residual, "residual", (m, n), dt)
    _like(out, "out", (m, n), dt)
    _like(z_out, "z_out", (m, n), dt)
    _workspace_ok(workspace)
    call = _Call(stream, x=x, w=w, bias=bias, residual=residual, group_offsets=group_offsets, out=out, z_out=z_out,
                 workspace=workspace)
    with call.scope:
        workspace = call.workspace(workspace, "mc2_linear_act_workspace_size", m, k, n, groups)
        if out is None:
            out = call.empty((m, n), dt)
        if need_z and z_out is None:
            z_out = call.empty((m, n), dt)
        _check(_lib.mc2_linear_act(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), m, k, n,
                                   _ptr(group_offsets), groups, _TORCH_DT[dt], act, out.data_ptr(), _ptr(z_out),
                                   _ptr(workspace), _bytes(workspace), call.handle))
    return out, z_out


def mc2_linear_act_grad(dout: torch.Tensor, x: torch.Tensor, w: torch.Tensor, z: Optional[torch.Tensor] = None, *,
                        act: int = MC2_ACT_NONE, group_offsets: Optional[torch.Tensor] = None, need_dx: bool = True,
                        need_dw: bool = True, need_dbias: bool = False, dx: Optional[torch.Tensor] = None,
                        dw: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dw, dbias) of mc2_linear_act, each None unless wanted (need_*, or given); z is its
    pre-activation (not needed with MC2_ACT_NONE).  The residual's gradient is dout itself."""
    m, k, n, groups = _linear_sizes(x, w, group_offsets)
    dt = x.dtype
    bias_shape = (groups, n) if groups else (n,)
    _needed(dout, "dout", (m, n), dt)
    if act != MC2_ACT_NONE:
        _needed(z, "z", (m, n), dt)
    else:
        _like(z, "z", (m, n), dt)
    _like(dx, "dx", (m, k), dt)
    _like(dw, "dw", w.shape, dt)
    _like(dbias, "dbias", bias_shape, dt)
    _workspace_ok(workspace)
    call = _Call(stream, dout=dout, x=x, w=w, z=z, group_offsets=group_offsets, dx=dx, dw=dw, dbias=dbias,
                 workspace=workspace)
    with call.scope:
        workspace = call.workspace(workspace, "mc2_linear_act_grad_workspace_size", m, k, n, groups)
        if need_dx and dx is None:
            dx = call.empty((m, k), dt)
        if need_dw and dw is None:
            dw = call.empty(w.shape, dt)
        if need_dbias and dbias is None:
            dbias = call.empty(bias_shape, dt)
        _check(_lib.mc2_linear_act_grad(dout.data_ptr(), _ptr(z), x.data_ptr(), w.data_ptr(), m, k, n,
                                        _ptr(group_offsets), groups, _TORCH_DT[dt], act, _ptr(dx), _ptr(dw),
                                        _ptr(dbias), _ptr(workspace), _bytes(workspace), call.handle))
    return dx, dw, dbias


# ------------------------------------------------------------------ tokens by expert
def mc2_moe_permute(x: torch.Tensor, expert_ids: torch.Tensor, experts: int, *, out: Optional[torch.Tensor] = None,
                    row_map: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Rows of x (tokens, h) for every choice expert_ids[t][j] (int32), sorted by expert and then by
    t * top + j: returns (out (tokens * top, h), row_map (tokens, top) int32, offsets (experts + 1)
    int32).  Ids outside [0, experts) are dropped: row_map -1; out's last rows are then 0."""
    tokens, h = _tensor(x, "x", 2)
    _half(x, "x")
    top = _tensor(expert_ids, "expert_ids", 2)[1]
    _needed(expert_ids, "expert_ids", (tokens, top), torch.int32)
    _like(out, "out", (tokens * top, h), x.dtype)
    _like(row_map, "row_map", (tokens, top), torch.int32)
    _like(offsets, "offsets", (experts + 1,), torch.int32)
    _workspace_ok(workspace)
    call = _Call(stream, x=x, expert_ids=expert_ids, out=out, row_map=row_map, offsets=offsets, workspace=workspace)
    with call.scope:
        workspace = call.workspace(workspace, "mc2_moe_permute_workspace_size", tokens, top, experts)
        if out is None:
            out = call.empty((tokens * top, h), x.dtype)
        if row_map is None:
            row_map = call.empty((tokens, top), torch.int32)
        if offsets is None:
            offsets = call.empty((experts + 1,), torch.int32)
        _check(_lib.mc2_moe_permute(x.data_ptr(), expert_ids.data_ptr(), tokens, top, h, experts, _TORCH_DT[x.dtype],
                                    out.data_ptr(), row_map.data_ptr(), offsets.data_ptr(), _ptr(workspace),
                                    _bytes(workspace), call.handle))
    return out, row_map, offsets


def mc2_moe_unpermute(y: torch.Tensor, row_map: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum over j of weights[t][j] * y[row_map[t][j]] (weights (tokens, top) fp32, or None
    for 1).  Without weights it is also mc2_moe_permute's gradient."""
    rows, h = _tensor(y, "y", 2)
    _half(y, "y")
    tokens, top = _tensor(row_map, "row_map", 2)
    _needed(row_map, "row_map", (tokens, top), torch.int32)
    _like(weights, "weights", (tokens, top), torch.float32)
    _like(out, "out", (tokens, h), y.dtype)
    call = _Call(stream, y=y, row_map=row_map, weights=weights, out=out)
    with call.scope:
        if out is None:
            out = call.empty((tokens, h), y.dtype)
        _check(_lib.mc2_moe_unpermute(y.data_ptr(), row_map.data_ptr(), _ptr(weights), tokens, top, h, rows,
                                      _TORCH_DT[y.dtype], out.data_ptr(), call.handle))
    return out


def mc2_moe_unpermute_grad(dout: torch.Tensor, y: torch.Tensor, row_map: torch.Tensor,
                           weights: Optional[torch.Tensor] = None, *, need_dweights: bool = True,
                           dy: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None, stream=None
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(dy, dweights) of mc2_moe_unpermute for a row_map that mc2_moe_permute gave."""
    rows, h = _tensor(y, "y", 2)
    _half(y, "y")
    tokens, top = _tensor(row_map, "row_map", 2)
    _needed(row_map, "row_map", (tokens, top), torch.int32)
    _needed(dout, "dout", (tokens, h), y.dtype)
    _like(weights, "weights", (tokens, top), torch.float32)
    _like(dy, "dy", (rows, h), y.dtype)
    _like(dweights, "dweights", (tokens, top), torch.float32)
    call = _Call(stream, dout=dout, y=y, row_map=row_map, weights=weights, dy=dy, dweights=dweights)
    with call.scope:
        if dy is None:
            dy = call.empty((rows, h), y.dtype)
        if need_dweights and dweights is None:
            dweights = call.empty((tokens, top), torch.float32)
        _check(_lib.mc2_moe_unpermute_grad(dout.data_ptr(), y.data_ptr(), row_map.data_ptr(), _ptr(weights), tokens,
                                           top, h, rows, _TORCH_DT[y.dtype], dy.data_ptr(), _ptr(dweights),
                                           call.handle))
    return dy, dweights


__all__ = ["MC2_ACT_NONE", "MC2_ACT_RELU", "MC2_ACT_GELU", "MC2_ACT_GELU_TANH", "MC2_ACT_SILU",
           "mc2_add_rms_norm", "mc2_add_rms_norm_grad", "mc2_linear_act", "mc2_linear_act_grad", "mc2_moe_permute",
           "mc2_moe_unpermute", "mc2_moe_unpermute_grad"]
