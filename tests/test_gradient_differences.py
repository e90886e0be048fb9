"""Gradients of the linear and of the norm, element by element against central differences of the forward formulas
in 64 bits; and, on the CPU, that the bounds tell a gradient with a term missing from the right one.

Bounds: the result rounds once (U |ref|).  The linear's products read dz rounded to 16 bits: U |dz| |w| (|dz| |x|),
and everything in fp32 is within 1e-5 of the same sums.  A difference of step d is off by d^2 / 6 times the third
derivative, below 1e-7 of the sums for d = 1e-4, and by 1e-16 / d = 1e-12 of the loss's terms.
"""
import pytest
import torch

from layer_ref import ACTS, U, act, check, norm, rand

EPS, STEP, U16 = 1e-6, 1e-4, U["bf16"]
M, K, N = 6, 24, 40


def linear_case(name):
    """x, w and dout, and z as z_out would hold it: gradients are taken there."""
    x, w, dout, z = rand(1, M, K), rand(2, N, K, std=K ** -0.5), rand(3, M, N), rand(4, M, N, std=1.5)
    if name == "relu":  # away from its corner
        z = torch.where(z.abs() < 0.05, torch.full_like(z, 0.5), z)
    return x, w, dout, z


def linear_differences(x, w, dout, z, name):
    """(dx, dw, dbias) of sum(dout act(z + what the argument adds to it)), one element at a time."""
    xd, wd, dd, zd = (t.double() for t in (x, w, dout, z))

    def slope_of(change):  # change (..., M, N): z's change for a unit of each element
        f = lambda s: (act(zd + s * STEP * change, name)[0] * dd).sum((-1, -2))
        return (f(1) - f(-1)) / (2 * STEP)

    eye_m, eye_n = torch.eye(M).double(), torch.eye(N).double()
    dx = slope_of(torch.einsum("im,nj->ijmn", eye_m, wd))
    dw = slope_of(torch.einsum("in,mj->ijmn", eye_n, xd))
    db = slope_of(eye_n[:, None, :].expand(N, M, N))
    return dx, dw, db


def linear_bounds(x, w, dout, z, refs):
    # |dz| of the elements: slopes are below 1.13
    dz = 1.13 * dout.double().abs()
    e = U16 + 1e-5
    sizes = dz @ w.double().abs(), dz.t() @ x.double().abs(), dz.sum(0)
    return [U16 * r.abs() + (e if i < 2 else 1e-5) * s for i, (r, s) in enumerate(zip(refs, sizes))]


def norm_case():
    s, w, dout, dsum = rand(11, 3, 48), rand(12, 48), rand(13, 3, 48), rand(14, 3, 48)
    return s, w, dout, dsum


def norm_differences(s, w, dout, dsum):
    sd, wd, dd, ds = (t.double() for t in (s, w, dout, dsum))

    def loss(sv, wv):
        y = sv / torch.sqrt((sv * sv).mean(-1, keepdim=True) + EPS) * wv
        return (y * dd + sv * ds).sum((-1, -2))

    rows, h = s.shape
    one = torch.eye(rows * h).double().view(rows, h, rows, h) * STEP
    dx = (loss(sd + one, wd) - loss(sd - one, wd)) / (2 * STEP)
    one = torch.eye(h).double()[:, None, :] * STEP
    return dx, (loss(sd, wd + one) - loss(sd, wd - one)) / (2 * STEP)


def norm_bounds(s, w, dout, dsum, refs):
    _, rstd, _ = norm(s, None, w, EPS)
    r, g, a = rstd[:, None], (dout.double() * w.double()).abs(), s.double().abs()
    terms = r * (g + a * r * r * (g * a).mean(1, keepdim=True)) + dsum.double().abs()
    return U16 * refs[0].abs() + 1e-5 * terms, U16 * refs[1].abs() + 1e-5 * (dout.double().abs() * a * r).sum(0)


def outside(got, ref, bound):
    return int((~((got - ref).abs() <= bound)).sum())


@pytest.mark.parametrize("name", ACTS)
def test_bounds_reject_a_linear_gradient_with_a_mistake(name):
    x, w, dout, z = linear_case(name)
    refs = linear_differences(x, w, dout, z, name)
    bounds = linear_bounds(x, w, dout, z, refs)
    zd, dd = z.double(), dout.double()

    def gradients(slope):
        dz = dd * slope
        return dz @ w.double(), dz.t() @ x.double(), dz.sum(0)

    for got, ref, bound in zip(gradients(act(zd, name)[1]), refs, bounds):
        assert outside(got, ref, bound) == 0  # the formula itself
    wrong = [torch.zeros_like(zd), act(zd, name)[1] * 1.02]
    if name != "none":
        wrong.append(torch.ones_like(zd))
        # without z times the factor's derivative (relu: with a leak)
        wrong.append(act(zd, name)[0] / zd if name != "relu" else torch.where(zd > 0, 1.0, 0.05).double())
    for slope in wrong:
        for got, ref, bound in zip(gradients(slope), refs, bounds):
            assert outside(got, ref, bound) > 0


def test_bounds_reject_a_norm_gradient_with_a_mistake():
    s, w, dout, dsum = norm_case()
    refs = norm_differences(s, w, dout, dsum)
    bounds = norm_bounds(s, w, dout, dsum, refs)
    sd, g, ds = s.double(), dout.double() * w.double(), dsum.double()
    r = (1 / torch.sqrt((sd * sd).mean(1) + EPS))[:, None]
    mean = sd * r * r * (g * sd).mean(1, keepdim=True)
    dw = (dout.double() * sd * r).sum(0)
    assert outside(r * (g - mean) + ds, refs[0], bounds[0]) == 0 and outside(dw, refs[1], bounds[1]) == 0
    for got in (r * g + ds, r * (g - mean), g - mean + ds, r * (dout.double() - mean) + ds, torch.zeros_like(sd)):
        assert outside(got, refs[0], bounds[0]) > 0
    for got in ((dout.double() * sd).sum(0), dw * w.double(), torch.zeros_like(dw)):
        assert outside(got, refs[1], bounds[1]) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ACTS)
def test_linear_gradient(name):
    import comm_matmul_tensor_amd as mc2
    x, w, dout, z = linear_case(name)
    got = mc2.mc2_linear_act_grad(dout.cuda(), x.cuda(), w.cuda(), z.cuda(), act=ACTS.index(name), need_dbias=True)
    refs = linear_differences(x, w, dout, z, name)
    for g, r, b, what in zip(got, refs, linear_bounds(x, w, dout, z, refs), ("dx", "dw", "dbias")):
        check(g, r, b, what)


@pytest.mark.gpu
def test_norm_gradient():
    import comm_matmul_tensor_amd as mc2
    s, w, dout, dsum = norm_case()
    _, _, _, rstd = mc2.mc2_add_rms_norm(s.cuda(), w.cuda(), eps=EPS, need_rstd=True)
    got = mc2.mc2_add_rms_norm_grad(dout.cuda(), s.cuda(), w.cuda(), rstd, dsum.cuda())
    refs = norm_differences(s, w, dout, dsum)
    for g, r, b, what in zip(got, refs, norm_bounds(s, w, dout, dsum, refs), ("dx", "dweight")):
        check(g, r, b, what)
