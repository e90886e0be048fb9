"""The feed-forward operators on the CPU: the library exports what include/mc2_layer.h declares, the
binding refuses mismatched tensors, and the C ABI refuses bad arguments, all before any device work."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import comm_matmul_tensor_amd as mc2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mc2_layer.h")
bf, f16, f32, i32, i8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int8
lib = ctypes.CDLL(mc2.LIB_PATH)
A, NULL, ODD = ctypes.c_void_p(0x10000), None, ctypes.c_void_p(0x10008)
OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_UNSUPPORTED, ERR_WORKSPACE, _, _, ERR_ALIGN = range(9)
F16, BF16, I8, I32, F8 = 1, 2, 3, 4, 5
I = ctypes.c_int64


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*mc2_status\s+(mc2_\w+)\s*\(", src, re.M)))


def test_exports_every_declared_symbol():
    names = declared()
    assert len(names) == 11, names
    for n in names:
        assert hasattr(lib, n), n
    for n in names:
        if not n.endswith("_workspace_size"):
            assert callable(getattr(mc2, n)) and n in mc2.__all__


def test_header_is_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "mc2_layer.h"\nint main(void) { return (int)MC2_ACT_NONE; }\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", f"-I{ROOT}/include", "-c", str(src), "-o",
                        str(tmp_path / "use.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_activation_codes_match_the_header():
    src = open(HEADER).read()
    for name in ("NONE", "RELU", "GELU", "GELU_TANH", "SILU"):
        assert int(re.search(rf"MC2_ACT_{name}\s*=\s*(\d+)", src).group(1)) == getattr(mc2, f"MC2_ACT_{name}")


# ------------------------------------------------------------------ the binding
@pytest.mark.parametrize("args,kwargs,exc,msg", [
    ((z(4, 64), z(63)), {}, ValueError, "weight has shape"),
    ((z(4, 64), z(64, dtype=f16)), {}, TypeError, "weight has dtype"),
    ((z(4, 64, dtype=f32), z(64, dtype=f32)), {}, TypeError, "float16 or bfloat16"),
    ((z(4, 64), z(64), z(4, 65)), {}, ValueError, "residual has shape"),
    ((z(4, 64), z(64)), dict(out_dtype=torch.uint8), TypeError, "out_dtype"),
    ((z(4, 64), z(64)), dict(out_dtype=f16), TypeError, "out_dtype"),
    ((z(4, 64), z(64)), dict(out_dtype=i8, group=128), ValueError, "group"),
    ((z(4, 256), z(256)), dict(group=128), ValueError, "group"),
    ((z(4, 256), z(256)), dict(out_dtype=i8, group=64), ValueError, "group"),
    ((z(4, 64), z(64)), dict(scale_out=z(4, 1, dtype=f32)), ValueError, "scale_out"),
    ((z(4, 64), z(64)), dict(out_dtype=i8, scale_out=z(4, 2, dtype=f32)), ValueError, "scale_out has shape"),
    ((z(4, 64), z(64)), dict(rstd_out=z(4)), TypeError, "rstd_out has dtype"),
    ((z(4, 64), z(64)), dict(out=z(4, 65)), ValueError, "out has shape"),
    ((z(4, 64), z(64)), dict(sum_out=z(3, 64)), ValueError, "sum_out has shape"),
    ((z(4, 128)[:, :64], z(64)), {}, ValueError, "x must be contiguous"),
    ((z(4, 64), z(64)), {}, ValueError, "must be a device tensor"),
    ((None, z(64)), {}, TypeError, "x must be a torch.Tensor"),
])
def test_norm_binding(args, kwargs, exc, msg):
    with pytest.raises(exc, match=msg):
        mc2.mc2_add_rms_norm(*args, **kwargs)


@pytest.mark.parametrize("args,kwargs,exc,msg", [
    ((z(4, 63), z(4, 64), z(64), z(4, dtype=f32)), {}, ValueError, "dout has shape"),
    ((z(4, 64), z(4, 64), z(64), z(4)), {}, TypeError, "rstd has dtype"),
    ((z(4, 64), z(4, 64), z(64), z(5, dtype=f32)), {}, ValueError, "rstd has shape"),
    ((z(4, 64), z(4, 64), z(64), z(4, dtype=f32), z(4, 64, dtype=f16)), {}, TypeError, "dsum has dtype"),
    ((z(4, 64), z(4, 64), z(64), None), {}, ValueError, "rstd is required"),
    ((z(4, 64), z(4, 64), z(64), z(4, dtype=f32)), dict(workspace=z(4, 4)), ValueError, "workspace"),
    ((z(4, 64), z(4, 64), z(64), z(4, dtype=f32)), {}, ValueError, "must be a device tensor"),
])
def test_norm_grad_binding(args, kwargs, exc, msg):
    with pytest.raises(exc, match=msg):
        mc2.mc2_add_rms_norm_grad(*args, **kwargs)


OFF = torch.zeros(4, dtype=i32)


@pytest.mark.parametrize("args,kwargs,exc,msg", [
    ((z(4, 64), z(32, 63)), {}, ValueError, "w has shape"),
    ((z(4, 64), z(32, 64, dtype=f16)), {}, TypeError, "w has dtype"),
    ((z(4, 64), z(3, 32, 64)), {}, ValueError, "w must be 2-D"),
    ((z(4, 64), z(32, 64)), dict(group_offsets=OFF), ValueError, "w must be 3-D"),
    ((z(4, 64), z(2, 32, 64)), dict(group_offsets=OFF), ValueError, "w has shape"),
    ((z(4, 64), z(3, 32, 64)), dict(group_offsets=OFF.long()), TypeError, "group_offsets has dtype"),
    ((z(4, 64), z(3, 32, 64)), dict(group_offsets=OFF[:1]), ValueError, "at least 2"),
    ((z(4, 64), z(32, 64), z(31)), {}, ValueError, "bias has shape"),
    ((z(4, 64), z(3, 32, 64), z(32)), dict(group_offsets=OFF), ValueError, "bias has shape"),
    ((z(4, 64), z(32, 64), None, z(4, 31)), {}, ValueError, "residual has shape"),
    ((z(4, 64), z(32, 64)), dict(out=z(4, 33)), ValueError, "out has shape"),
    ((z(4, 64), z(32, 64)), dict(z_out=z(4, 32, dtype=f16)), TypeError, "z_out has dtype"),
    ((z(4, 64), z(64, 32).t()), {}, ValueError, "w must be contiguous"),
    ((z(4, 64), z(32, 64)), {}, ValueError, "must be a device tensor"),
    ((z(4, 64, dtype=f32), z(32, 64, dtype=f32)), {}, TypeError, "float16 or bfloat16"),
])
def test_linear_binding(args, kwargs, exc, msg):
    with pytest.raises(exc, match=msg):
        mc2.mc2_linear_act(*args, **kwargs)


@pytest.mark.parametrize("args,kwargs,exc,msg", [
    ((z(4, 31), z(4, 64), z(32, 64)), {}, ValueError, "dout has shape"),
    ((z(4, 32), z(4, 64), z(32, 64)), dict(act=mc2.MC2_ACT_GELU), ValueError, "z is required"),
    ((z(4, 32), z(4, 64), z(32, 64), z(4, 33)), dict(act=mc2.MC2_ACT_GELU), ValueError, "z has shape"),
    ((z(4, 32), z(4, 64), z(32, 64)), dict(dx=z(4, 63)), ValueError, "dx has shape"),
    ((z(4, 32), z(4, 64), z(32, 64)), dict(dw=z(64, 32)), ValueError, "dw has shape"),
    ((z(4, 32), z(4, 64), z(32, 64)), dict(dbias=z(4)), ValueError, "dbias has shape"),
    ((z(4, 32), z(4, 64), z(32, 64)), {}, ValueError, "must be a device tensor"),
])
def test_linear_grad_binding(args, kwargs, exc, msg):
    with pytest.raises(exc, match=msg):
        mc2.mc2_linear_act_grad(*args, **kwargs)


IDS = torch.zeros((4, 2), dtype=i32)


def test_moe_binding():
    cases = [
        (mc2.mc2_moe_permute, (z(4, 8), IDS[:3], 4), {}, ValueError, "expert_ids has shape"),
        (mc2.mc2_moe_permute, (z(4, 8), IDS.long(), 4), {}, TypeError, "expert_ids has dtype"),
        (mc2.mc2_moe_permute, (z(4, 8), IDS, 4), dict(out=z(4, 8)), ValueError, "out has shape"),
        (mc2.mc2_moe_permute, (z(4, 8), IDS, 4), dict(offsets=torch.zeros(4, dtype=i32)), ValueError, "offsets has shape"),
        (mc2.mc2_moe_permute, (z(4, 8), IDS, 4), {}, ValueError, "must be a device tensor"),
        (mc2.mc2_moe_unpermute, (z(8, 8), IDS, z(4, 2)), {}, TypeError, "weights has dtype"),
        (mc2.mc2_moe_unpermute, (z(8, 8), IDS, z(4, 3, dtype=f32)), {}, ValueError, "weights has shape"),
        (mc2.mc2_moe_unpermute, (z(8, 8), IDS), dict(out=z(8, 8)), ValueError, "out has shape"),
        (mc2.mc2_moe_unpermute, (z(8, 8), IDS), {}, ValueError, "must be a device tensor"),
        (mc2.mc2_moe_unpermute_grad, (z(3, 8), z(8, 8), IDS), {}, ValueError, "dout has shape"),
        (mc2.mc2_moe_unpermute_grad, (z(4, 8, dtype=f16), z(8, 8), IDS), {}, TypeError, "dout has dtype"),
        (mc2.mc2_moe_unpermute_grad, (z(4, 8), z(8, 8), IDS), dict(dy=z(4, 8)), ValueError, "dy has shape"),
        (mc2.mc2_moe_unpermute_grad, (z(4, 8), z(8, 8), IDS), {}, ValueError, "must be a device tensor"),
    ]
    for fn, args, kwargs, exc, msg in cases:
        with pytest.raises(exc, match=msg):
            fn(*args, **kwargs)


# ------------------------------------------------------------------ the C ABI
def call(name, *args):
    return getattr(lib, name)(*args)


def test_norm_abi():
    def norm(x=A, res=A, w=A, rows=4, h=256, dt=BF16, eps=1e-6, out=A, odt=BF16, scale=NULL, group=0, s=A, rstd=A):
        return call("mc2_add_rms_norm", x, res, w, I(rows), I(h), dt, ctypes.c_float(eps), out, odt, scale, I(group), s,
                    rstd, NULL)

    assert norm(rows=-1) == ERR_SHAPE and norm(rows=1 << 24) == ERR_SHAPE
    assert norm(h=0) == ERR_SHAPE and norm(h=(1 << 24) + 1) == ERR_SHAPE
    assert norm(dt=0, odt=0) == ERR_DTYPE and norm(odt=F16) == ERR_DTYPE and norm(odt=I32) == ERR_DTYPE
    assert norm(eps=-1e-6) == ERR_SHAPE and norm(eps=float("nan")) == ERR_SHAPE and norm(eps=float("inf")) == ERR_SHAPE
    assert norm(group=128) == ERR_SHAPE and norm(odt=I8, scale=A, group=64) == ERR_SHAPE
    assert norm(odt=I8, scale=A, group=128, h=200) == ERR_SHAPE
    assert norm(odt=I8) == ERR_NULL and norm(odt=F8) == ERR_NULL
    assert norm(x=NULL) == ERR_NULL and norm(w=NULL) == ERR_NULL and norm(out=NULL) == ERR_NULL
    for k in ("x", "res", "w", "out", "s", "rstd"):
        assert norm(**{k: ODD}) == ERR_ALIGN, k
    assert norm(rows=0, x=NULL, res=NULL, out=NULL, s=NULL, rstd=NULL) == OK

    def grad(dout=A, dsum=A, s=A, w=A, rstd=A, rows=4, h=256, dt=BF16, dx=A, dw=A, ws=A, n=1 << 20):
        return call("mc2_add_rms_norm_grad", dout, dsum, s, w, rstd, I(rows), I(h), dt, dx, dw, ws, ctypes.c_size_t(n),
                    NULL)

    for k in ("dout", "s", "w", "rstd", "dx", "dw"):
        assert grad(**{k: NULL}) == ERR_NULL, k
        assert grad(**{k: ODD}) == ERR_ALIGN, k
    assert grad(h=0) == ERR_SHAPE and grad(rows=-1) == ERR_SHAPE and grad(dt=I8) == ERR_DTYPE
    need = ctypes.c_size_t(0)
    assert call("mc2_add_rms_norm_grad_workspace_size", I(4), I(256), ctypes.byref(need)) == OK and need.value == 4096
    assert grad(n=need.value - 1) == ERR_WORKSPACE and grad(ws=NULL) == ERR_WORKSPACE and grad(ws=ODD) == ERR_ALIGN
    assert call("mc2_add_rms_norm_grad_workspace_size", I(4), I(256), NULL) == ERR_NULL
    assert call("mc2_add_rms_norm_grad_workspace_size", I(4), I(0), ctypes.byref(need)) == ERR_SHAPE


def test_linear_abi():
    big = 1 << 40

    def fwd(x=A, w=A, bias=A, res=A, m=64, k=128, n=256, off=NULL, g=0, dt=BF16, act=0, out=A, zo=A, ws=A, nb=big):
        return call("mc2_linear_act", x, w, bias, res, I(m), I(k), I(n), off, I(g), dt, act, out, zo, ws,
                    ctypes.c_size_t(nb), NULL)

    assert fwd(m=-1) == ERR_SHAPE and fwd(m=1 << 24) == ERR_SHAPE
    assert fwd(k=0) == ERR_SHAPE and fwd(k=(1 << 21) + 1) == ERR_SHAPE
    assert fwd(n=0) == ERR_SHAPE and fwd(n=(1 << 21) + 1) == ERR_SHAPE
    assert fwd(g=-1) == ERR_SHAPE and fwd(g=4097, off=A) == ERR_SHAPE
    assert fwd(g=4096, off=A, n=1 << 18) == ERR_SHAPE and fwd(g=4096, off=A, k=1 << 18) == ERR_SHAPE
    assert fwd(g=3) == ERR_NULL and fwd(off=A) == ERR_SHAPE
    assert fwd(dt=0) == ERR_DTYPE and fwd(act=5) == ERR_UNSUPPORTED and fwd(act=-1) == ERR_UNSUPPORTED
    for k in ("x", "w", "out"):
        assert fwd(**{k: NULL}) == ERR_NULL, k
    for k in ("x", "w", "bias", "res", "out", "zo"):
        assert fwd(**{k: ODD}) == ERR_ALIGN, k
    assert fwd(m=0, x=NULL, w=NULL, out=NULL, ws=NULL, nb=0) == OK
    need = ctypes.c_size_t(0)
    assert call("mc2_linear_act_workspace_size", I(64), I(4096), I(256), I(0), ctypes.byref(need)) == OK
    assert need.value > 0  # a split contraction
    assert fwd(k=4096, nb=need.value - 1) == ERR_WORKSPACE and fwd(k=4096, ws=NULL) == ERR_WORKSPACE
    assert fwd(k=4096, ws=ODD) == ERR_ALIGN
    assert call("mc2_linear_act_workspace_size", I(1), I(4096), I(4096), I(0), ctypes.byref(need)) == OK
    assert need.value == 0
    assert call("mc2_linear_act_workspace_size", I(1), I(1), I(1), I(0), NULL) == ERR_NULL

    def grad(dout=A, zi=A, x=A, w=A, m=64, k=128, n=256, off=NULL, g=0, dt=BF16, act=2, dx=A, dw=A, db=A, ws=A, nb=big):
        return call("mc2_linear_act_grad", dout, zi, x, w, I(m), I(k), I(n), off, I(g), dt, act, dx, dw, db, ws,
                    ctypes.c_size_t(nb), NULL)

    assert grad(dout=NULL) == ERR_NULL and grad(zi=NULL) == ERR_NULL
    assert grad(x=NULL) == ERR_NULL and grad(w=NULL) == ERR_NULL
    for k in ("dout", "zi", "x", "w", "dx", "dw", "db"):
        assert grad(**{k: ODD}) == ERR_ALIGN, k
    assert grad(m=1 << 24) == ERR_SHAPE and grad(dt=F8) == ERR_DTYPE and grad(act=9) == ERR_UNSUPPORTED
    assert grad(g=2) == ERR_NULL and grad(nb=16) == ERR_WORKSPACE and grad(ws=NULL) == ERR_WORKSPACE
    assert call("mc2_linear_act_grad_workspace_size", I(64), I(128), I(256), I(0), ctypes.byref(need)) == OK
    assert need.value >= 64 * 256 * 2


def test_moe_abi():
    big = 1 << 40

    def permute(x=A, ids=A, t=64, top=2, h=128, e=8, dt=BF16, out=A, m=A, off=A, ws=A, nb=big):
        return call("mc2_moe_permute", x, ids, I(t), I(top), I(h), I(e), dt, out, m, off, ws, ctypes.c_size_t(nb), NULL)

    assert permute(t=-1) == ERR_SHAPE and permute(t=(1 << 23) + 1) == ERR_SHAPE
    assert permute(top=0) == ERR_SHAPE and permute(t=1 << 20, top=1 << 12) == ERR_SHAPE
    assert permute(h=0) == ERR_SHAPE and permute(e=0) == ERR_SHAPE and permute(e=4097) == ERR_SHAPE
    assert permute(dt=0) == ERR_DTYPE
    for k in ("x", "ids", "out", "m", "off"):
        assert permute(**{k: NULL}) == ERR_NULL, k
        assert permute(**{k: ODD}) == ERR_ALIGN, k
    need = ctypes.c_size_t(1)
    assert call("mc2_moe_permute_workspace_size", I(16), I(2), I(8), ctypes.byref(need)) == OK and need.value == 0
    assert call("mc2_moe_permute_workspace_size", I(9000), I(2), I(8), ctypes.byref(need)) == OK and need.value > 0
    assert permute(t=9000, ws=NULL) == ERR_WORKSPACE and permute(t=9000, nb=need.value - 1) == ERR_WORKSPACE
    assert call("mc2_moe_permute_workspace_size", I(16), I(2), I(8), NULL) == ERR_NULL

    def unpermute(y=A, m=A, w=A, t=64, top=2, h=128, rows=128, dt=BF16, out=A):
        return call("mc2_moe_unpermute", y, m, w, I(t), I(top), I(h), I(rows), dt, out, NULL)

    assert unpermute(rows=-1) == ERR_SHAPE and unpermute(rows=1 << 31) == ERR_SHAPE and unpermute(h=0) == ERR_SHAPE
    assert unpermute(dt=I8) == ERR_DTYPE
    for k in ("y", "m", "out"):
        assert unpermute(**{k: NULL}) == ERR_NULL, k
    for k in ("y", "m", "w", "out"):
        assert unpermute(**{k: ODD}) == ERR_ALIGN, k
    assert unpermute(t=0, y=NULL, m=NULL, out=NULL) == OK

    def grad(dout=A, y=A, m=A, w=A, t=64, top=2, h=128, rows=128, dt=BF16, dy=A, dw=A):
        return call("mc2_moe_unpermute_grad", dout, y, m, w, I(t), I(top), I(h), I(rows), dt, dy, dw, NULL)

    for k in ("dout", "y", "m"):
        assert grad(**{k: NULL}) == ERR_NULL, k
    assert grad(dy=NULL, dw=NULL) == ERR_NULL
    for k in ("dout", "y", "m", "w", "dy", "dw"):
        assert grad(**{k: ODD}) == ERR_ALIGN, k
    assert grad(top=0) == ERR_SHAPE and grad(dt=0) == ERR_DTYPE
