"""mc2_linear_act's slopes at infinity.

x of one column and w = 1 make dx the slope rounded to 16 bits, for dout = 1.
"""
import math

import pytest
import torch

from layer_ref import ACTS, DT, U, act, check, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


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
