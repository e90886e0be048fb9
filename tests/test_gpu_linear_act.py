"""mc2_linear_act and its gradient against their formulas in 64 bits, dense and by groups of rows.

Bounds, element by element: a product of k terms accumulated in fp32 in any
order is within (k + 4) roundings of sum |x| |w| + |bias|; an activation moves
that by at most its largest slope (below 1.13) and adds its own error
(layer_ref.ACT_ERR); the residual's addition and the output round once each.
The gradients' products read dz rounded to 16 bits: one more unit roundoff of
|dz| @ |w| (|dz|^T @ |x|).
"""
import math

import pytest
import torch

from layer_ref import ACT_ERR, ACTS, DT, EPS32, TINY, U, act, check, rand, rounded, spans

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


def forward_ref(x, w, bias, residual, name, groups):
    """(out, z, bound of out, bound of z); groups: [(g, begin, end)] or None."""
    m, k = x.shape
    n = w.shape[-2]
    z = torch.zeros((m, n), dtype=torch.float64)
    ez = torch.zeros((m, n), dtype=torch.float64)
    for g, a, b in groups or [(None, 0, m)]:
        wg = w.double() if g is None else w[g].double()
        z[a:b] = x[a:b].double() @ wg.T
        ez[a:b] = x[a:b].double().abs() @ wg.abs().T
        if bias is not None:
            bg = bias.double() if g is None else bias[g].double()
            z[a:b] += bg
            ez[a:b] += bg.abs()
    ez = (k + 4) * EPS32 * ez
    out, _ = act(z, name)
    eo = 1.13 * ez + (0 if name in ("none", "relu") else ACT_ERR * (1 + z.abs()))
    if residual is not None:
        eo = eo + EPS32 * (out.abs() + residual.double().abs())
        out = out + residual.double()
    return out, z, eo, ez


def run_forward(mc2, seed, m, k, n, dtype, name, bias, residual, offsets=None, keep_z=True):
    G = 0 if offsets is None else len(offsets) - 1
    x = rand(seed, m, k, dtype=dtype)
    w = rand(seed + 1, *((G, n, k) if G else (n, k)), std=1.5 * k ** -0.5, dtype=dtype)
    b = rand(seed + 2, *((G, n) if G else (n,)), std=0.5, dtype=dtype) if bias else None
    r = rand(seed + 3, m, n, dtype=dtype) if residual else None
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    out, z = mc2.mc2_linear_act(x.cuda(), w.cuda(), None if b is None else b.cuda(), None if r is None else r.cuda(),
                                act=ACTS.index(name), group_offsets=off, need_z=keep_z)
    ref, zr, eo, ez = forward_ref(x, w, b, r, name, None if offsets is None else spans(offsets, m))
    assert out.dtype == DT[dtype]
    check(out, ref, rounded(ref, dtype) * (1 + U[dtype]) + eo, "out")
    if keep_z:
        check(z, zr, rounded(zr, dtype) * (1 + U[dtype]) + ez, "z")
    else:
        assert z is None


# few rows (one fragment or two), one tile and several, ragged everywhere, one of everything
SIZES = [(1, 1, 1), (1, 8, 16), (1, 4096, 1792), (2, 33, 7), (5, 264, 100), (16, 512, 4100), (17, 1000, 65),
         (32, 2049, 33), (33, 64, 64), (33, 63, 65), (64, 4096, 256), (100, 40, 1000), (129, 136, 127), (128, 8, 8),
         (257, 129, 131), (300, 200, 520), (517, 1792, 384), (1, 5, 3000), (256, 1, 256), (700, 72, 1), (1000, 576, 777)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward_sizes(mc2, m, k, n, dtype):
    print(f"linear m={m} k={k} n={n} {dtype}", flush=True)
    run_forward(mc2, m + k + n, m, k, n, dtype, "gelu", True, True)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [3, 40, 200])
@pytest.mark.parametrize("bias,residual,keep_z", [(False, False, False), (True, False, True), (False, True, False)])
def test_forward_epilogues(mc2, name, dtype, m, bias, residual, keep_z):
    run_forward(mc2, 11, m, 328, 296, dtype, name, bias, residual, keep_z=keep_z)


@pytest.mark.parametrize("m,k,n", [(4096, 256, 4096), (2048, 320, 2048), (4100, 200, 3850)])
def test_forward_large_tiles(mc2, m, k, n):
    """Outputs of many tiles: the 256- and 128-row tiles, their edges, even and odd numbers of K steps."""
    print(f"linear m={m} k={k} n={n}", flush=True)
    run_forward(mc2, 5, m, k, n, "bf16", "silu", True, True)


GROUPS = [
    (64, [0, 64]),
    (300, [0, 100, 100, 290]),                # an empty group, rows of no group
    (700, [0, 1, 257, 513, 700]),             # one row, whole tiles, a partial tile
    (500, [0, 0, 0, 500, 500]),
    (40, [0, 3, 9, 9, 14, 15, 30, 33]),
    (130, [0, 0]),                            # no row in any group
    (1000, [0] + [i * 1000 // 70 for i in range(1, 71)]),   # more groups than lanes
    (90, [0, 50, 20, 200, 60]),               # descending and past the end: 50, 50, 90, 90
    (3, [0, 1, 2, 3]),
]


@pytest.mark.parametrize("m,offsets", GROUPS)
@pytest.mark.parametrize("k,n", [(256, 128), (200, 264), (77, 39)])
def test_forward_groups(mc2, m, offsets, k, n):
    print(f"groups m={m} k={k} n={n} offsets={offsets[:8]}", flush=True)
    run_forward(mc2, 21, m, k, n, "bf16", "silu", True, True, offsets)
    run_forward(mc2, 22, m, k, n, "f16", "none", False, False, offsets, keep_z=False)


# outputs of 193 to 256 tiles of 96 x 64, 128 x 64 and 96 x 128, with partial ones at both edges; 64 x 64 whole
# and with K in parts
MIDDLE = [(381, 150, 4090), (509, 77, 4091), (761, 456, 4088), (250, 136, 4088), (70, 2056, 1030), (512, 512, 4096)]


@pytest.mark.parametrize("m,k,n", MIDDLE)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward_middle_tiles(mc2, m, k, n, dtype):
    print(f"linear m={m} k={k} n={n} {dtype}", flush=True)
    run_forward(mc2, 26, m, k, n, dtype, "gelu_tanh", True, True)


def many_groups(m, groups):
    """Ranges of 0 to 60 rows, every fifth one empty, one end out of order, rows left over."""
    g = torch.Generator().manual_seed(groups)
    sizes = torch.randint(0, 61, (groups,), generator=g)
    sizes[::5] = 0
    offsets = [0] + (sizes.cumsum(0) * (m - 9) // sizes.sum()).tolist()
    offsets[groups // 2] = offsets[groups // 3]
    return offsets


def test_forward_many_groups(mc2):
    run_forward(mc2, 24, 3000, 72, 136, "bf16", "silu", True, True, many_groups(3000, 700))
    run_forward(mc2, 25, 9000, 64, 520, "f16", "none", True, False, many_groups(9000, 129))


def test_forward_groups_large_tiles(mc2):
    run_forward(mc2, 23, 2500, 192, 2048, "bf16", "gelu", True, False, [0, 700, 1500, 1501, 2470])


# ------------------------------------------------------------------ gradients
def grad_ref(dout, z, x, w, name, groups):
    m, k = x.shape
    n = w.shape[-2]
    slope = act(z.double(), name)[1] if name != "none" else torch.ones((m, n), dtype=torch.float64)
    dz = dout.double() * slope
    ez = (0 if name in ("none", "relu") else ACT_ERR) * dout.double().abs() * (1 + z.double().abs()) ** 3 + \
        2 * EPS32 * dz.abs()
    G = 1 if groups is None else w.shape[0]
    wg = (w[None] if groups is None else w).double()
    dx, sx = torch.zeros((m, k), dtype=torch.float64), torch.zeros((m, k), dtype=torch.float64)
    dw, sw = torch.zeros((G, n, k), dtype=torch.float64), torch.zeros((G, n, k), dtype=torch.float64)
    db, sb = torch.zeros((G, n), dtype=torch.float64), torch.zeros((G, n), dtype=torch.float64)
    return dz, ez, wg, (dx, sx), (dw, sw), (db, sb), groups or [(0, 0, m)]


def run_grad(mc2, seed, m, k, n, dtype, name, offsets=None):
    G = 0 if offsets is None else len(offsets) - 1
    x, dout, z = rand(seed, m, k, dtype=dtype), rand(seed + 1, m, n, dtype=dtype), rand(seed + 2, m, n, std=1.5, dtype=dtype)
    w = rand(seed + 3, *((G, n, k) if G else (n, k)), std=n ** -0.5, dtype=dtype)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    dx, dw, db = mc2.mc2_linear_act_grad(dout.cuda(), x.cuda(), w.cuda(), None if name == "none" else z.cuda(),
                                         act=ACTS.index(name), group_offsets=off, need_dbias=True)
    dz, ez, wg, (rx, sx), (rw, sw), (rb, sb), groups = grad_ref(dout, z, x, w, name,
                                                                None if offsets is None else spans(offsets, m))
    u = U[dtype]
    # |error of the dz the products read|: its own and its rounding
    e16 = ez + (0 if name == "none" else 1) * (u * dz.abs() + TINY[dtype])
    for g, a, b in groups:
        xa = x[a:b].double()
        rx[a:b] = dz[a:b] @ wg[g]
        sx[a:b] = e16[a:b] @ wg[g].abs() + (n + 4) * EPS32 * (dz[a:b].abs() * (1 + u)) @ wg[g].abs()
        rw[g] = dz[a:b].T @ xa
        sw[g] = e16[a:b].T @ xa.abs() + (b - a + 4) * EPS32 * (dz[a:b].abs() * (1 + u)).T @ xa.abs()
        rb[g] = dz[a:b].sum(0)
        sb[g] = ez[a:b].sum(0) + (b - a + 8) * EPS32 * dz[a:b].abs().sum(0)
    if not G:
        rw, sw, rb, sb = rw[0], sw[0], rb[0], sb[0]
    check(dx, rx, rounded(rx, dtype) * (1 + u) + sx, "dx")
    check(dw, rw, rounded(rw, dtype) * (1 + u) + sw, "dw")
    check(db, rb, rounded(rb, dtype) * (1 + u) + sb, "dbias")
    return dx, dw, db


@pytest.mark.parametrize("m,k,n", [(1, 1, 1), (1, 64, 128), (2, 7, 9), (16, 520, 40), (33, 63, 65), (100, 129, 200),
                                   (129, 256, 127), (300, 520, 264), (517, 136, 72), (64, 1, 300), (1000, 77, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_grad_sizes(mc2, m, k, n, dtype, name):
    print(f"linear_grad m={m} k={k} n={n} {dtype} {name}", flush=True)
    run_grad(mc2, m + k + n, m, k, n, dtype, name)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_grad_activations(mc2, name, dtype):
    run_grad(mc2, 31, 190, 200, 168, dtype, name)


@pytest.mark.parametrize("m,k,n", [(256, 2048, 4096), (4096, 2304, 130), (200, 4096, 4096), (4096, 128, 128)])
def test_grad_large_tiles(mc2, m, k, n):
    """Large and small outputs of either product: every tile, and a split contraction."""
    print(f"linear_grad m={m} k={k} n={n}", flush=True)
    run_grad(mc2, 32, m, k, n, "bf16", "silu")


@pytest.mark.parametrize("m,n,k", MIDDLE)
def test_grad_middle_tiles(mc2, m, n, k):
    """dx (m, k), and dw (n, k) by as many rows of it, with tiles under 128 x 128."""
    print(f"linear_grad m={m} k={k} n={n}", flush=True)
    run_grad(mc2, 38, m, k, n, "bf16", "silu")
    run_grad(mc2, 39, n, k, m, "f16", "none")


@pytest.mark.parametrize("m,offsets", GROUPS)
@pytest.mark.parametrize("k,n", [(128, 256), (200, 264), (77, 39)])
def test_grad_groups(mc2, m, offsets, k, n):
    print(f"grad groups m={m} k={k} n={n} offsets={offsets[:8]}", flush=True)
    run_grad(mc2, 33, m, k, n, "bf16", "silu", offsets)
    run_grad(mc2, 34, m, k, n, "f16", "none", offsets)


def test_grad_many_groups(mc2):
    run_grad(mc2, 36, 3000, 72, 136, "bf16", "silu", many_groups(3000, 700))
    run_grad(mc2, 37, 9000, 64, 520, "f16", "gelu", many_groups(9000, 129))


def test_grad_groups_large_tiles(mc2):
    run_grad(mc2, 35, 2500, 1024, 2048, "bf16", "gelu", [0, 700, 1500, 1501, 2470])


def test_grad_differences(mc2):
    """dx, dw and dbias against central differences of the forward formula in 64 bits."""
    m, k, n = 6, 24, 40
    for name in ACTS:
        x, w, b, dout = rand(41, m, k), rand(42, n, k, std=k ** -0.5), rand(43, n), rand(44, m, n)
        _, z = mc2.mc2_linear_act(x.cuda(), w.cuda(), b.cuda(), act=ACTS.index(name), need_z=True)
        if name == "relu":  # away from its corner
            dout = torch.where(z.cpu().float().abs() < 0.05, torch.zeros_like(dout), dout)
        dx, dw, db = mc2.mc2_linear_act_grad(dout.cuda(), x.cuda(), w.cuda(), z, act=ACTS.index(name), need_dbias=True)

        def loss(xv, wv, bv):
            return (act(xv @ wv.T + bv, name)[0] * dout.double()).sum()

        d, base = 1e-5, [x.double(), w.double(), b.double()]
        for i, got in enumerate((dx, dw, db)):
            v = rand(45 + i, *base[i].shape).double()
            hi, lo = list(base), list(base)
            hi[i], lo[i] = base[i] + d * v, base[i] - d * v
            num = (loss(*hi) - loss(*lo)) / (2 * d)
            # z, dz and the result are each rounded to 8 bits; slopes change by at most 1.2 |dz|
            got = got.cpu().double()
            tol = (4 * U["bf16"] * (got.abs() + 2.0) * v.abs()).sum()
            assert abs(num - (got * v).sum()) <= tol, (name, i)


def test_only_what_is_wanted(mc2):
    x, w, dout = rand(51, 70, 96).cuda(), rand(52, 80, 96).cuda(), rand(53, 70, 80).cuda()
    full = mc2.mc2_linear_act_grad(dout, x, w, need_dbias=True)
    for wanted in ((True, False, False), (False, True, False), (False, False, True), (True, True, False)):
        got = mc2.mc2_linear_act_grad(dout, x, w, need_dx=wanted[0], need_dw=wanted[1], need_dbias=wanted[2])
        for on, a, b in zip(wanted, got, full):
            assert (a is not None) == on
            if on:
                assert torch.equal(a, b)


def test_no_rows(mc2):
    x, w, b = rand(54, 0, 96).cuda(), rand(55, 80, 96).cuda(), rand(56, 80).cuda()
    out, z = mc2.mc2_linear_act(x, w, b, act=mc2.MC2_ACT_SILU, need_z=True)
    assert out.shape == (0, 80) and z.shape == (0, 80)
    dw, db = torch.full_like(w, 7.0), torch.full_like(b, 7.0)
    dx, dw, db = mc2.mc2_linear_act_grad(out, x, w, z, act=mc2.MC2_ACT_SILU, need_dbias=True, dw=dw, dbias=db)
    assert dx.shape == (0, 96) and torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    w3 = rand(57, 3, 80, 96).cuda()
    assert mc2.mc2_linear_act(x, w3, group_offsets=off)[0].shape == (0, 80)
    _, dw, _ = mc2.mc2_linear_act_grad(out, x, w3, group_offsets=off)
    assert dw.shape == w3.shape and torch.count_nonzero(dw) == 0


def test_residual_in_place(mc2):
    for m in (5, 150):
        x, w, r = rand(58, m, 128).cuda(), rand(59, 136, 128).cuda(), rand(60, m, 136).cuda()
        want, _ = mc2.mc2_linear_act(x, w, residual=r, act=mc2.MC2_ACT_GELU)
        got, _ = mc2.mc2_linear_act(x, w, residual=r, act=mc2.MC2_ACT_GELU, out=r)
        assert got is r and torch.equal(got, want)


def test_nan_and_infinity_stay_in_their_rows(mc2):
    """A NaN or an infinity in one row of x reaches that row's outputs only, in every path."""
    for m, offsets in ((8, None), (24, None), (200, None), (200, [0, 90, 150])):
        x = rand(61, m, 136)
        clean = x.clone()
        x[3, 5], x[m - 1, 135] = float("nan"), float("inf")
        w = rand(62, *((2, 72, 136) if offsets else (72, 136)))
        off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
        got = mc2.mc2_linear_act(x.cuda(), w.cuda(), group_offsets=off)[0].cpu()
        ref = mc2.mc2_linear_act(clean.cuda(), w.cuda(), group_offsets=off)[0].cpu()
        others = [i for i in range(m) if i not in (3, m - 1)]
        assert torch.equal(got[others], ref[others])
        assert torch.isnan(got[3]).all()
        if offsets is None:
            assert not torch.isfinite(got[m - 1].float()).any()
        else:
            assert torch.count_nonzero(got[150:]) == 0  # rows of no group are not read


def test_activations_of_extremes(mc2):
    """z of 0, large values and infinities through every activation (x = z, w = 1)."""
    z = torch.tensor([0.0, 1e-30, -1e-30, 3.0, -3.0, 20.0, -20.0, 200.0, -200.0, 3e4, -3e4, 1e38, -1e38])
    for name in ACTS:
        for m in (1, 40):
            x = z.bfloat16()[None].T.contiguous()
            x = x if m == 1 else x.repeat(4, 1)
            out, _ = mc2.mc2_linear_act(x.cuda(), torch.ones((1, 1)).bfloat16().cuda(), act=ACTS.index(name))
            zr = x.double()
            if name == "gelu_tanh":
                zr = zr.clamp(min=-1e12)  # z^3 leaves fp32's range there; the limit is 0
            ref = act(zr, name)[0]
            check(out, ref, rounded(ref, "bf16") * 1.01 + ACT_ERR * (1 + zr.abs().clamp(max=64.0)), name)


def test_slopes_of_extremes(mc2):
    """act'(z) at 0, large values and the largest (dout = 1, w = 1: dx is the slope)."""
    z = torch.tensor([0.0, 1e-30, -1e-30, 3.0, -3.0, 20.0, -20.0, 200.0, -200.0, 3e4, -3e4, 1e38, -1e38]).bfloat16()
    for name in ACTS[1:]:
        one = torch.ones((13, 1)).bfloat16().cuda()
        dx, _, _ = mc2.mc2_linear_act_grad(one, one, one[:1], z[:, None].contiguous().cuda(), act=ACTS.index(name))
        zr = z.double()[:, None].clamp(min=-1e6, max=1e6)  # the slopes' limits are reached long before
        ref = act(zr, name)[1]
        check(dx, ref, rounded(ref, "bf16") * 1.01 + ACT_ERR * (1 + zr.abs().clamp(max=8.0)) ** 3, name)


def test_offsets_past_32_bits(mc2):
    """Operands of more than 2^31 elements: the last rows and columns of the result."""
    k = 65536
    w = torch.zeros((33000, k), dtype=torch.bfloat16, device="cuda")
    tail = rand(63, 8, k, std=k ** -0.5)
    w[-8:] = tail.cuda()
    for m in (2, 48):  # the product of few rows, and a split one of tiles
        x = rand(64, m, k)
        out, _ = mc2.mc2_linear_act(x.cuda(), w)
        ref = x.double() @ tail.double().T
        size = x.double().abs() @ tail.double().abs().T
        check(out[:, -8:], ref, rounded(ref, "bf16") + (k + 4) * EPS32 * size, "out")
    # x (m, k) and its gradient likewise: rows past the range, and a contraction over them for dw
    x = w
    w2 = rand(65, 24, k, std=k ** -0.5)
    out, _ = mc2.mc2_linear_act(x, w2.cuda())
    ref = tail.double() @ w2.double().T
    check(out[-8:], ref, rounded(ref, "bf16") + (k + 4) * EPS32 * (tail.double().abs() @ w2.double().abs().T), "out")
    dout = torch.zeros((33000, 24), dtype=torch.bfloat16, device="cuda")
    dtail = rand(66, 8, 24)
    dout[-8:] = dtail.cuda()
    dx, dw, _ = mc2.mc2_linear_act_grad(dout, x, w2.cuda())
    ref = dtail.double() @ w2.double()
    check(dx[-8:], ref, rounded(ref, "bf16") + 30 * EPS32 * (dtail.double().abs() @ w2.double().abs()), "dx")
    ref = dtail.double().T @ tail.double()
    check(dw, ref, rounded(ref, "bf16") + 33000 * EPS32 * (dtail.double().abs().T @ tail.double().abs()), "dw")


def test_same_bits_and_other_stream(mc2):
    for m, offsets in ((4, None), (400, None), (700, [0, 300, 300, 650])):
        x, dout = rand(67, m, 320).cuda(), rand(68, m, 264).cuda()
        w = rand(69, *((3, 264, 320) if offsets else (264, 320))).cuda()
        off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
        a, z = mc2.mc2_linear_act(x, w, act=mc2.MC2_ACT_SILU, group_offsets=off, need_z=True)
        ga = mc2.mc2_linear_act_grad(dout, x, w, z, act=mc2.MC2_ACT_SILU, group_offsets=off, need_dbias=True)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        b, zb = mc2.mc2_linear_act(x, w, act=mc2.MC2_ACT_SILU, group_offsets=off, need_z=True, stream=st)
        gb = mc2.mc2_linear_act_grad(dout, x, w, z, act=mc2.MC2_ACT_SILU, group_offsets=off, need_dbias=True, stream=st)
        st.synchronize()
        for p, q in zip((a, z, *ga), (b, zb, *gb)):
            assert torch.equal(p, q)


def test_graph_replay(mc2):
    """A norm, a linear, experts and their rows' return in one captured graph, replayed on new inputs."""
    x = rand(70, 96, 256).cuda()
    wn, w = rand(71, 256).cuda(), rand(72, 4, 64, 256, std=1 / 16).cuda()
    w1 = rand(73, 256, 256, std=1 / 16).cuda()
    ids = torch.randint(0, 4, (96, 2), generator=torch.Generator().manual_seed(74), dtype=torch.int32).cuda()

    def step():
        y, _, s, _ = mc2.mc2_add_rms_norm(x, wn, x)
        a, _ = mc2.mc2_linear_act(y, w1, residual=s, act=mc2.MC2_ACT_GELU)
        p, row_map, off = mc2.mc2_moe_permute(a, ids, 4)
        e, _ = mc2.mc2_linear_act(p, w, act=mc2.MC2_ACT_SILU, group_offsets=off)
        return mc2.mc2_moe_unpermute(e, row_map)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(rand(80 + i, 96, 256).cuda())
        ids.copy_(torch.randint(-1, 4, (96, 2), generator=torch.Generator().manual_seed(90 + i), dtype=torch.int32).cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())
        torch.cuda.synchronize()
