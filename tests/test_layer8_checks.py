"""The router and the 8-bit operators on the CPU: the library exports what include/mc2_layer8.h declares, the binding
refuses mismatched tensors, and the C ABI refuses bad arguments, all before any device work."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import comm_matmul_tensor_amd as mc2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mc2_layer8.h")
bf, f16, f32, i32, i8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int8
lib = ctypes.CDLL(mc2.LIB_PATH)
A, NULL, ODD = ctypes.c_void_p(0x10000), None, ctypes.c_void_p(0x10008)
OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_UNSUPPORTED, ERR_WORKSPACE, _, _, ERR_ALIGN = range(9)
F32, F16, BF16, I8 = 0, 1, 2, 3
I, SZ = ctypes.c_int64, ctypes.c_size_t


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*mc2_status\s+(mc2_\w+)\s*\(", src, re.M)))


def test_exports_every_declared_symbol():
    names = declared()
    assert len(names) == 8, names
    for n in names:
        assert hasattr(lib, n), n
        if not n.endswith("_workspace_size"):
            assert callable(getattr(mc2, n)) and n in mc2.__all__


def test_header_is_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "mc2_layer8.h"\nint main(void) { return (int)MC2_SCORE_SOFTMAX; }\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", f"-I{ROOT}/include", "-c", str(src), "-o",
                        str(tmp_path / "use.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_score_codes_match_the_header():
    src = open(HEADER).read()
    for name in ("SOFTMAX", "SIGMOID"):
        assert int(re.search(rf"MC2_SCORE_{name}\s*=\s*(\d+)", src).group(1)) == getattr(mc2, f"MC2_SCORE_{name}")


# ------------------------------------------------------------------ the binding
L = z(4, 16, dtype=f32)
IDS, W = z(4, 2, dtype=i32), z(4, 2, dtype=f32)
S4 = z(4, dtype=f32)
X8, W8 = z(4, 64, dtype=i8), z(32, 64, dtype=i8)
S32 = z(32, dtype=f32)
OFF = z(4, dtype=i32)
W16 = z(32, 64)
D = z(4, 32)
XS, ZS, Z8 = z(4, 1, dtype=f32), z(4, 1, dtype=f32), z(4, 32, dtype=i8)
GELU = dict(act=mc2.MC2_ACT_GELU)

CASES = [
    (mc2.mc2_moe_route, (L.double(), 2), {}, TypeError, "logits must be float32"),
    (mc2.mc2_moe_route, (L[0], 2), {}, ValueError, "logits must be 2-D"),
    (mc2.mc2_moe_route, (L, 2, z(15, dtype=f32)), {}, ValueError, "bias has shape"),
    (mc2.mc2_moe_route, (L, 2, z(16)), {}, TypeError, "bias has dtype"),
    (mc2.mc2_moe_route, (L, 2), dict(expert_ids=IDS.long()), TypeError, "expert_ids has dtype"),
    (mc2.mc2_moe_route, (L, 3), dict(weights=W), ValueError, "weights has shape"),
    (mc2.mc2_moe_route, (L.t(), 2), {}, ValueError, "logits must be contiguous"),
    (mc2.mc2_moe_route, (L, 2), {}, ValueError, "must be a device tensor"),
    (mc2.mc2_moe_route_grad, (z(4, 3, dtype=f32), L, IDS), {}, ValueError, "dweights has shape"),
    (mc2.mc2_moe_route_grad, (z(4, 2), L, IDS), {}, TypeError, "dweights has dtype"),
    (mc2.mc2_moe_route_grad, (W, L, IDS[:3]), {}, ValueError, "expert_ids has shape"),
    (mc2.mc2_moe_route_grad, (W, L, IDS), dict(dlogits=z(4, 16)), TypeError, "dlogits has dtype"),
    (mc2.mc2_moe_route_grad, (W, L, IDS), {}, ValueError, "must be a device tensor"),
    (mc2.mc2_quant_rows, (L,), {}, TypeError, "float16 or bfloat16"),
    (mc2.mc2_quant_rows, (W16,), dict(group=64), ValueError, "group must be 0 or 128"),
    (mc2.mc2_quant_rows, (W16,), dict(codes=X8), ValueError, "codes has shape"),
    (mc2.mc2_quant_rows, (W16,), dict(scale=S32), ValueError, "scale has shape"),
    (mc2.mc2_quant_rows, (W16,), dict(scale=z(32, 2, dtype=f32), group=128), ValueError, "scale has shape"),
    (mc2.mc2_quant_rows, (z(8, 128)[:, :64],), {}, ValueError, "x must be contiguous"),
    (mc2.mc2_quant_rows, (W16,), {}, ValueError, "must be a device tensor"),
    (mc2.mc2_quant_rows, (torch.zeros((), dtype=bf),), {}, ValueError, "last dimension"),
    (mc2.mc2_dequant_rows, (W16, S32), {}, TypeError, "codes must be int8"),
    (mc2.mc2_dequant_rows, (X8, S4), {}, ValueError, "scale has shape"),
    (mc2.mc2_dequant_rows, (X8, XS), dict(dtype=f32), TypeError, "float16 or bfloat16"),
    (mc2.mc2_dequant_rows, (X8, XS), dict(out=z(4, 63)), ValueError, "out has shape"),
    (mc2.mc2_dequant_rows, (X8, None), {}, ValueError, "scale is required"),
    (mc2.mc2_dequant_rows, (X8, XS), {}, ValueError, "must be a device tensor"),
    (mc2.mc2_linear_i8, (z(4, 64), S4, W8, S32), {}, TypeError, "x must be int8"),
    (mc2.mc2_linear_i8, (X8, S4, W16, S32), {}, TypeError, "w has dtype"),
    (mc2.mc2_linear_i8, (X8, S4, z(32, 63, dtype=i8), S32), {}, ValueError, "w has shape"),
    (mc2.mc2_linear_i8, (X8, z(5, dtype=f32), W8, S32), {}, ValueError, "x_scale has shape"),
    (mc2.mc2_linear_i8, (X8, z(4, 2, dtype=f32), W8, S32), {}, ValueError, "x_scale has shape"),
    (mc2.mc2_linear_i8, (X8, S4, W8, z(32)), {}, TypeError, "w_scale has dtype"),
    (mc2.mc2_linear_i8, (X8, None, W8, S32), {}, ValueError, "x_scale is required"),
    (mc2.mc2_linear_i8, (X8, S4, W8, S32), dict(group_offsets=OFF), ValueError, "w must be 3-D"),
    (mc2.mc2_linear_i8, (X8, S4, z(3, 32, 64, dtype=i8), S32), dict(group_offsets=OFF), ValueError, "w_scale has shape"),
    (mc2.mc2_linear_i8, (X8, S4, z(3, 32, 64, dtype=i8), z(3, 32, dtype=f32)), dict(group_offsets=OFF.long()), TypeError,
     "group_offsets has dtype"),
    (mc2.mc2_linear_i8, (X8, S4, W8, S32, z(31)), {}, ValueError, "bias has shape"),
    (mc2.mc2_linear_i8, (X8, S4, W8, S32, z(32), z(4, 32, dtype=f16)), {}, TypeError, "bias has dtype"),
    (mc2.mc2_linear_i8, (X8, S4, W8, S32, None, z(4, 31)), {}, ValueError, "residual has shape"),
    (mc2.mc2_linear_i8, (X8, S4, W8, S32), dict(dtype=f32), TypeError, "float16 or bfloat16"),
    (mc2.mc2_linear_i8, (X8, S4, W8, S32), dict(out=D, dtype=f16), TypeError, "out has dtype"),
    (mc2.mc2_linear_i8, (X8, S4, W8, S32), dict(workspace=z(4, 4)), ValueError, "workspace"),
    (mc2.mc2_linear_i8, (X8, S4, z(64, 32, dtype=i8).t(), S32), {}, ValueError, "w must be contiguous"),
    (mc2.mc2_linear_i8, (X8, S4, W8, S32), {}, ValueError, "must be a device tensor"),
    (mc2.mc2_linear_act_grad_i8, (D, W16[:4], XS, W16), {}, TypeError, "x must be int8"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16.float()), {}, TypeError, "w must be float16"),
    (mc2.mc2_linear_act_grad_i8, (z(4, 31), X8, XS, W16), {}, ValueError, "dout has shape"),
    (mc2.mc2_linear_act_grad_i8, (D.half(), X8, XS, W16), {}, TypeError, "dout has dtype"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, z(4, 2, dtype=f32), W16), {}, ValueError, "x_scale has shape"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16), GELU, ValueError, "z is required"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16, Z8), GELU, ValueError, "z_scale is required"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16, D, ZS), GELU, TypeError, "z has dtype"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16, Z8, S4), GELU, ValueError, "z_scale has shape"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16), dict(dx=z(4, 63)), ValueError, "dx has shape"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16), dict(dw=z(64, 32)), ValueError, "dw has shape"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16), dict(dbias=z(4)), ValueError, "dbias has shape"),
    (mc2.mc2_linear_act_grad_i8, (D, X8, XS, W16), {}, ValueError, "must be a device tensor"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_binding(i):
    fn, args, kwargs, exc, msg = CASES[i]
    with pytest.raises(exc, match=msg):
        fn(*args, **kwargs)


# ------------------------------------------------------------------ the C ABI
def test_route_abi():
    def route(l=A, b=A, t=16, e=64, top=4, dt=F32, sc=0, g=1, tg=1, gt=1, rn=1, scale=1.0, ids=A, w=A):
        return lib.mc2_moe_route(l, b, I(t), I(e), I(top), dt, sc, I(g), I(tg), I(gt), rn, ctypes.c_float(scale), ids, w,
                                 NULL)

    assert route(t=-1) == ERR_SHAPE and route(t=(1 << 23) + 1) == ERR_SHAPE
    assert route(e=0) == ERR_SHAPE and route(e=4097) == ERR_SHAPE
    assert route(top=0) == ERR_SHAPE and route(top=65, e=128) == ERR_SHAPE and route(e=3) == ERR_SHAPE
    assert route(dt=I8) == ERR_DTYPE and route(sc=2) == ERR_UNSUPPORTED and route(sc=-1) == ERR_UNSUPPORTED
    assert route(g=0) == ERR_SHAPE and route(g=5) == ERR_SHAPE and route(g=128, e=128) == ERR_SHAPE
    assert route(g=8, tg=0) == ERR_SHAPE and route(g=8, tg=9) == ERR_SHAPE and route(tg=2) == ERR_SHAPE
    assert route(g=8, tg=2, gt=0) == ERR_SHAPE and route(g=8, tg=2, gt=3) == ERR_SHAPE
    assert route(g=64, tg=8, gt=2) == ERR_SHAPE and route(g=16, tg=1, top=5) == ERR_SHAPE
    assert route(scale=float("nan")) == ERR_SHAPE and route(scale=float("inf")) == ERR_SHAPE
    for k in ("l", "ids", "w"):
        assert route(**{k: NULL}) == ERR_NULL, k
    for k in ("l", "b", "ids", "w"):
        assert route(**{k: ODD}) == ERR_ALIGN, k
    assert route(t=0, l=NULL, b=NULL, ids=NULL, w=NULL) == OK

    def grad(dw=A, l=A, ids=A, t=16, e=64, top=4, dt=F32, sc=0, rn=1, scale=1.0, dl=A):
        return lib.mc2_moe_route_grad(dw, l, ids, I(t), I(e), I(top), dt, sc, rn, ctypes.c_float(scale), dl, NULL)

    assert grad(t=-1) == ERR_SHAPE and grad(e=4097) == ERR_SHAPE and grad(top=65, e=128) == ERR_SHAPE
    assert grad(dt=I8) == ERR_DTYPE and grad(sc=7) == ERR_UNSUPPORTED and grad(scale=float("nan")) == ERR_SHAPE
    for k in ("dw", "l", "ids", "dl"):
        assert grad(**{k: NULL}) == ERR_NULL, k
        assert grad(**{k: ODD}) == ERR_ALIGN, k
    assert grad(t=0, dw=NULL, l=NULL, ids=NULL, dl=NULL) == OK


def test_codes_abi():
    def quant(x=A, r=4, c=256, dt=BF16, g=0, q=A, s=A):
        return lib.mc2_quant_rows(x, I(r), I(c), dt, I(g), q, s, NULL)

    def back(q=A, s=A, r=4, c=256, g=0, act=0, dt=BF16, o=A):
        return lib.mc2_dequant_rows(q, s, I(r), I(c), I(g), act, dt, o, NULL)

    for fn, names in ((quant, ("x", "q", "s")), (back, ("q", "s", "o"))):
        assert fn(r=-1) == ERR_SHAPE and fn(r=1 << 24) == ERR_SHAPE
        assert fn(c=0) == ERR_SHAPE and fn(c=(1 << 24) + 1) == ERR_SHAPE
        assert fn(dt=F32) == ERR_DTYPE and fn(g=64) == ERR_SHAPE and fn(g=-128) == ERR_SHAPE
        for k in names:
            assert fn(**{k: NULL}) == ERR_NULL, k
            assert fn(**{k: ODD}) == ERR_ALIGN, k
        assert fn(r=0, **{k: NULL for k in names}) == OK
    assert back(act=5) == ERR_UNSUPPORTED and back(act=-1) == ERR_UNSUPPORTED


def test_linear_i8_abi():
    big = 1 << 40

    def fwd(x=A, xs=A, w=A, ws=A, bias=A, res=A, m=64, k=128, n=256, off=NULL, g=0, dt=BF16, act=0, out=A, wsp=A, nb=big):
        return lib.mc2_linear_i8(x, xs, w, ws, bias, res, I(m), I(k), I(n), off, I(g), dt, act, out, wsp, SZ(nb), NULL)

    assert fwd(m=-1) == ERR_SHAPE and fwd(m=1 << 24) == ERR_SHAPE
    assert fwd(k=0) == ERR_SHAPE and fwd(k=1 << 17) == ERR_SHAPE
    assert fwd(n=0) == ERR_SHAPE and fwd(n=(1 << 21) + 1) == ERR_SHAPE
    assert fwd(g=-1) == ERR_SHAPE and fwd(g=4097, off=A) == ERR_SHAPE and fwd(g=4096, off=A, n=1 << 18) == ERR_SHAPE
    assert fwd(g=3) == ERR_NULL and fwd(off=A) == ERR_SHAPE
    assert fwd(dt=F32) == ERR_DTYPE and fwd(act=5) == ERR_UNSUPPORTED and fwd(act=-1) == ERR_UNSUPPORTED
    for k in ("x", "xs", "w", "ws", "out"):
        assert fwd(**{k: NULL}) == ERR_NULL, k
    for k in ("x", "xs", "w", "ws", "bias", "res", "out"):
        assert fwd(**{k: ODD}) == ERR_ALIGN, k
    assert fwd(m=0, x=NULL, xs=NULL, w=NULL, ws=NULL, out=NULL, wsp=NULL, nb=0) == OK
    need = SZ(0)
    size = lib.mc2_linear_i8_workspace_size
    assert size(I(64), I(8192), I(256), I(0), ctypes.byref(need)) == OK and need.value > 0  # a split contraction
    assert fwd(k=8192, nb=need.value - 1) == ERR_WORKSPACE and fwd(k=8192, wsp=NULL) == ERR_WORKSPACE
    assert fwd(k=8192, wsp=ODD) == ERR_ALIGN
    assert size(I(64), I(102), I(256), I(0), ctypes.byref(need)) == OK and need.value >= 112 * (64 + 256)  # rows to copy
    assert size(I(1), I(4096), I(4096), I(0), ctypes.byref(need)) == OK and need.value == 0
    assert size(I(1), I(1), I(1), I(0), NULL) == ERR_NULL
    assert size(I(1), I(1 << 17), I(1), I(0), ctypes.byref(need)) == ERR_SHAPE

    def grad(dout=A, zi=A, zs=A, x=A, xs=A, xa=0, w=A, m=64, k=128, n=256, off=NULL, g=0, dt=BF16, act=2, dx=A, dw=A, db=A,
             wsp=A, nb=big):
        return lib.mc2_linear_act_grad_i8(dout, zi, zs, x, xs, xa, w, I(m), I(k), I(n), off, I(g), dt, act, dx, dw, db, wsp,
                                          SZ(nb), NULL)

    for k in ("dout", "zi", "zs", "x", "xs", "w"):
        assert grad(**{k: NULL}) == ERR_NULL, k
        assert grad(**{k: ODD}) == ERR_ALIGN, k
    for k in ("dx", "dw", "db"):
        assert grad(**{k: ODD}) == ERR_ALIGN, k
    assert grad(m=1 << 24) == ERR_SHAPE and grad(k=(1 << 21) + 1) == ERR_SHAPE and grad(dt=F32) == ERR_DTYPE
    assert grad(act=9) == ERR_UNSUPPORTED and grad(xa=5) == ERR_UNSUPPORTED and grad(xa=-1) == ERR_UNSUPPORTED
    assert grad(g=2) == ERR_NULL and grad(nb=16) == ERR_WORKSPACE and grad(wsp=NULL) == ERR_WORKSPACE
    size = lib.mc2_linear_act_grad_i8_workspace_size
    assert size(I(64), I(128), I(256), I(0), ctypes.byref(need)) == OK and need.value >= 64 * (256 + 128) * 2
    assert size(I(64), I(128), I(256), I(0), NULL) == ERR_NULL
    assert size(I(-1), I(128), I(256), I(0), ctypes.byref(need)) == ERR_SHAPE


def test_plan_hook():
    tile, splits = ctypes.c_int(), ctypes.c_int()
    plan = lib.mc2_testing_linear_i8_plan
    assert plan(I(1), I(4096), I(4096), I(0), ctypes.byref(tile), ctypes.byref(splits)) == OK and tile.value < 0
    assert plan(I(64), I(4096), I(4096), I(0), NULL, ctypes.byref(splits)) == ERR_NULL
    assert plan(I(64), I(1 << 17), I(4096), I(0), ctypes.byref(tile), ctypes.byref(splits)) == ERR_SHAPE


def test_keep_inf_is_for_groups_of_128():
    src = open(HEADER).read()
    assert re.search(r"MC2_KEEP_INF\s*=\s*1 << 16", src) and mc2.MC2_KEEP_INF == 1 << 16
    with pytest.raises(ValueError, match="keep_inf needs group 128"):
        mc2.mc2_quant_rows(W16, keep_inf=True)
    with pytest.raises(ValueError, match="must be a device tensor"):
        mc2.mc2_quant_rows(W16, group=128, keep_inf=True)
    flag = mc2.MC2_KEEP_INF
    for g in (flag, flag + 64, flag + 256, 2 * flag + 128, 128 - flag):
        assert lib.mc2_quant_rows(A, I(4), I(256), BF16, I(g), A, A, NULL) == ERR_SHAPE, g
    assert lib.mc2_quant_rows(NULL, I(0), I(256), BF16, I(flag + 128), NULL, NULL, NULL) == OK
    assert lib.mc2_quant_rows(A, I(4), I(256), F32, I(flag + 128), A, A, NULL) == ERR_DTYPE
    assert lib.mc2_dequant_rows(A, A, I(4), I(256), I(flag + 128), 0, BF16, A, NULL) == ERR_SHAPE


def test_keep_nan_is_for_a_score():
    assert re.search(r"MC2_SCORE_KEEP_NAN\s*=\s*1 << 16", open(HEADER).read()) and mc2.MC2_SCORE_KEEP_NAN == 1 << 16
    flag = mc2.MC2_SCORE_KEEP_NAN
    route = lambda sc, t=16: lib.mc2_moe_route(A if t else NULL, NULL, I(t), I(64), I(4), F32, sc, I(1), I(1), I(1), 1,
                                               ctypes.c_float(1.0), NULL, A, NULL)
    assert route(flag) == ERR_NULL and route(flag + 1) == ERR_NULL
    assert route(flag, 0) == OK and route(flag + 1, 0) == OK
    for sc in (flag + 2, flag - 1, 2 * flag, -flag, -flag + 1):
        assert route(sc) == ERR_UNSUPPORTED, sc
    assert lib.mc2_moe_route_grad(A, A, A, I(16), I(64), I(4), F32, flag, 1, ctypes.c_float(1.0), A, NULL) == ERR_UNSUPPORTED
