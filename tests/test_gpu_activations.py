"""mc2_linear_act's activations and slopes element by element over all of the 16-bit values near 0, and at infinity.

x of one column and w = 1 make z = x exactly, and dout = 1 and w = 1 make dx the slope rounded to 16 bits, so a
result's error is that of the activation and of one rounding.  Bounds, relative to the term that carries them:
Phi(-|z|) by its formula 1e-6; z^2 in fp32 and the exponential of it 3 roundings of z^2 / 2; the other products,
sums and reciprocals (exponential and reciprocal: 1 ulp) 16 roundings.  The tanh form's exponential is of
z (A + B z^2), 6 roundings of it, silu's of z, 2.
"""
import math

import pytest
import torch

from layer_ref import ACTS, DT, EPS32, U, act, check, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


def values(dtype, top):
    """Every value of the type with 2^-10 <= |z| <= top."""
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    a = v.double().abs()
    return v[(a >= 2.0 ** -10) & (a <= top)]


def relative(z, name):
    """Relative error of the activation's factor of z: Phi(z) or the sigmoid; its complement's is absolute."""
    if name == "gelu":
        return 1e-6 + (16 + 1.5 * z * z) * EPS32
    u = z if name == "silu" else math.sqrt(8 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3)
    return (16 + (2 if name == "silu" else 6) * u.abs()) * EPS32


def factor(z, name):
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5))  # torch.special.ndtr is 1 + erf, which cancels below 0
    return torch.sigmoid(z if name == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))


def factor_error(z, name):
    """Error of p = factor(z): on either side that of the smaller of p and 1 - p, and fp32's of p."""
    small = factor(-z.abs(), name)
    return relative(z, name) * small + 2 * EPS32 * factor(z, name)


# (up to where the results and the exponentials are normal fp32 numbers)
TOP = {"gelu": 12.5, "gelu_tanh": 9.0, "silu": 80.0}


@pytest.mark.parametrize("name", sorted(TOP))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_activation_of_every_value(mc2, name, dtype):
    v = values(dtype, TOP[name])
    z = v.double()
    ref = z * factor(z, name)
    bound = rounded(ref, dtype) * (1 + U[dtype]) + z.abs() * factor_error(z, name) + 2 * EPS32 * ref.abs()
    one = torch.ones((1, 1), dtype=DT[dtype]).cuda()
    out, _ = mc2.mc2_linear_act(v[:, None].cuda(), one, act=ACTS.index(name))  # many rows
    check(out[:, 0], ref, bound, "rows")
    out, _ = mc2.mc2_linear_act(one, v[:, None].cuda(), act=ACTS.index(name))  # one row
    check(out[0], ref, bound, "columns")


@pytest.mark.parametrize("name", sorted(TOP))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_slope_of_every_value(mc2, name, dtype):
    v = values(dtype, TOP[name])
    z = v.double()
    p = factor(z, name)
    if name == "gelu":
        term = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        steep = 1.0
    else:
        steep = 1.0 if name == "silu" else math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z)
        term = z * p * factor(-z, name) * steep
    ref = p + term
    # p (1 - p): 1 - p is formed from p, so p's own rounding counts in full where p is near 1
    bound = rounded(ref, dtype) * (1 + U[dtype]) + factor_error(z, name) + relative(z, name) * term.abs()
    if name != "gelu":
        bound = bound + z.abs() * p * steep * factor_error(z, name)
    one = torch.ones((v.numel(), 1), dtype=DT[dtype]).cuda()
    dx, _, _ = mc2.mc2_linear_act_grad(one, one, one[:1], v[:, None].cuda(), act=ACTS.index(name))
    check(dx[:, 0], ref, bound, "dx")


@pytest.mark.parametrize("name", ACTS[1:])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_slopes_at_infinity(mc2, name, dtype):
    """act'(+inf) = 1 and act'(-inf) = 0 and beside them the type's largest values; a NaN's slope is NaN (relu's 0)."""
    big = torch.finfo(DT[dtype]).max
    z = torch.tensor([math.inf, -math.inf, big, -big, 0.5, math.nan]).to(DT[dtype])[:, None]
    one = torch.ones((6, 1), dtype=DT[dtype]).cuda()
    dx, _, db = mc2.mc2_linear_act_grad(one, one, one[:1], z.cuda(), act=ACTS.index(name), need_dbias=True)
    dx = dx.cpu().double()[:, 0]
    assert dx[:4].tolist() == [1.0, 0.0, 1.0, 0.0]
    ref = act(z[4:5].double(), name)[1][0]
    check(dx[4:5], ref, 2 * rounded(ref, dtype), "0.5")
    assert dx[5] == 0.0 if name == "relu" else math.isnan(dx[5])


@pytest.mark.parametrize("name", ACTS[1:])
def test_gradient_of_a_saved_infinity(mc2, name):
    """A pre-activation past fp16's range has a finite output and is saved as an infinity: its gradient is finite too."""
    m, k, n = 40, 8, 24
    x, w = torch.ones((m, k)).half(), torch.full((n, k), 0.25).half()
    w[3] = -9000.0  # z = -72000
    w[5] = 9000.0
    out, z = mc2.mc2_linear_act(x.cuda(), w.cuda(), act=ACTS.index(name), need_z=True)
    assert torch.isneginf(z[:, 3]).all() and torch.isposinf(z[:, 5]).all()
    assert torch.count_nonzero(out[:, 3]) == 0
    dout = torch.full((m, n), 2.0 ** -12).half().cuda()
    dx, dw, db = mc2.mc2_linear_act_grad(dout, x.cuda(), w.cuda(), z, act=ACTS.index(name), need_dbias=True)
    zr = torch.full((n,), 2.0, dtype=torch.float64)
    zr[3], zr[5] = -1e3, 1e3
    slope = act(zr, name)[1]
    dz = slope * 2.0 ** -12
    u, err = U["f16"], 1e-5
    bound = lambda ref, size: rounded(ref, "f16") + (u + err) * size
    ref = torch.full((m, k), float(dz @ w[:, 0].double()), dtype=torch.float64)
    check(dx, ref, bound(ref, float(dz.abs() @ w[:, 0].double().abs())), "dx")
    ref = (m * dz)[:, None].expand(n, k)
    check(dw, ref, bound(ref, ref.abs()), "dw")
    check(db, m * dz, bound(m * dz, (m * dz).abs()), "dbias")
