"""mc2_linear_act_grad_i8 against its formulas in 64 bits of the values that the codes stand for.

Bounds as in test_gpu_linear_act.py, with one rounding more: xv = x_act(code scale) is rounded to 16 bits for its
product, as dz is (and code * scale rounds once in fp32 before an activation or a slope).
"""
import pytest
import torch

import layer8_ref as ref
from layer_ref import ACT_ERR, ACTS, DT, EPS32, TINY, U, act, check, rand, rounded, spans

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


def run(mc2, seed, m, k, n, dtype, name, x_name="none", offsets=None):
    G = 0 if offsets is None else len(offsets) - 1
    u = U[dtype]
    xc, xs = ref.codes(rand(seed, m, k, std=1.5, dtype=dtype), 128)
    zc, zs = ref.codes(rand(seed + 2, m, n, std=1.5, dtype=dtype), 128)
    dout = rand(seed + 1, m, n, dtype=dtype)
    w = rand(seed + 3, *((G, n, k) if G else (n, k)), std=n ** -0.5, dtype=dtype)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    zargs = () if name == "none" else (zc.cuda(), zs.cuda())
    dx, dw, db = mc2.mc2_linear_act_grad_i8(dout.cuda(), xc.cuda(), xs.cuda(), w.cuda(), *zargs, act=ACTS.index(name),
                                            x_act=ACTS.index(x_name), group_offsets=off, need_dbias=True)
    xr, zv = ref.values(xc, xs, 128), ref.values(zc, zs, 128)
    x = act(xr, x_name)[0]
    ex = EPS32 * 1.13 * xr.abs() + (0 if x_name in ("none", "relu") else ACT_ERR * (1 + xr.abs()))
    ex = ex + u * (x.abs() + ex) + TINY[dtype]
    slope = act(zv, name)[1] if name != "none" else torch.ones_like(zv)
    dz = dout.double() * slope
    # a slope changes by at most 1.2 |dz|, relu's (at exact zeros only) not at all
    ez = (0 if name in ("none", "relu") else ACT_ERR * (1 + zv.abs()) ** 3 + 1.2 * EPS32 * zv.abs()) * dout.double().abs() + \
        2 * EPS32 * dz.abs()
    e16 = ez + (0 if name == "none" else 1) * (u * dz.abs() + TINY[dtype])
    wg = (w if G else w[None]).double()
    shape = dict(dtype=torch.float64)
    rx, sx = torch.zeros((m, k), **shape), torch.zeros((m, k), **shape)
    rw, sw = torch.zeros(wg.shape, **shape), torch.zeros(wg.shape, **shape)
    rb, sb = torch.zeros(wg.shape[:2], **shape), torch.zeros(wg.shape[:2], **shape)
    for g, a, b in spans(offsets, m) if G else [(0, 0, m)]:
        d, xa, e = dz[a:b], x[a:b], e16[a:b]
        rx[a:b] = d @ wg[g]
        sx[a:b] = e @ wg[g].abs() + (n + 4) * EPS32 * (d.abs() * (1 + u)) @ wg[g].abs()
        rw[g] = d.T @ xa
        sw[g] = e.T @ (xa.abs() + ex[a:b]) + d.abs().T @ ex[a:b] + \
            (b - a + 4) * EPS32 * (d.abs() * (1 + u)).T @ (xa.abs() + ex[a:b])
        rb[g] = d.sum(0)
        sb[g] = ez[a:b].sum(0) + (b - a + 8) * EPS32 * d.abs().sum(0)
    if not G:
        rw, sw, rb, sb = rw[0], sw[0], rb[0], sb[0]
    check(dx, rx, rounded(rx, dtype) * (1 + u) + sx, "dx")
    check(dw, rw, rounded(rw, dtype) * (1 + u) + sw, "dw")
    check(db, rb, rounded(rb, dtype) * (1 + u) + sb, "dbias")


@pytest.mark.parametrize("m,k,n", [(1, 1, 1), (1, 64, 128), (2, 7, 9), (16, 520, 40), (33, 63, 65), (100, 129, 200),
                                   (129, 256, 127), (300, 520, 264), (517, 136, 72), (64, 1, 300), (1000, 77, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name,x_name", [("none", "gelu"), ("gelu", "none")])
def test_sizes(mc2, m, k, n, dtype, name, x_name):
    print(f"kept grad m={m} k={k} n={n} {dtype} {name} {x_name}", flush=True)
    run(mc2, m + k + n, m, k, n, dtype, name, x_name)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("x_name", ACTS)
def test_activations(mc2, name, x_name):
    run(mc2, 31, 90, 200, 168, "bf16", name, x_name)
    run(mc2, 32, 40, 130, 260, "f16", name, x_name)


@pytest.mark.parametrize("m,k,n", [(256, 2048, 4096), (4096, 2304, 130), (200, 4096, 4096)])
def test_larger_tiles(mc2, m, k, n):
    print(f"kept grad m={m} k={k} n={n}", flush=True)
    run(mc2, 33, m, k, n, "bf16", "silu", "silu")


GROUPS = [(64, [0, 64]), (300, [0, 100, 100, 290]), (700, [0, 1, 257, 513, 700]), (500, [0, 0, 0, 500, 500]),
          (130, [0, 0]), (90, [0, 50, 20, 200, 60]), (3, [0, 1, 2, 3])]


@pytest.mark.parametrize("m,offsets", GROUPS)
@pytest.mark.parametrize("k,n", [(128, 256), (200, 264), (77, 39)])
def test_groups(mc2, m, offsets, k, n):
    print(f"kept grad groups m={m} k={k} n={n} offsets={offsets[:8]}", flush=True)
    run(mc2, 34, m, k, n, "bf16", "silu", "none", offsets)
    run(mc2, 35, m, k, n, "f16", "none", "silu", offsets)


def test_against_the_16_bit_gradient(mc2):
    """The same bits as mc2_linear_act_grad on the codes' values, where those round nowhere else on the way."""
    for m, k, n, offsets in ((70, 200, 264, None), (300, 131, 77, None), (90, 128, 256, [0, 40, 40, 80])):
        G = 0 if offsets is None else len(offsets) - 1
        off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
        x = rand(41, m, k).cuda()
        w = rand(42, *((G, n, k) if G else (n, k))).cuda()
        dout = rand(43, m, n).cuda()
        xc, xs = mc2.mc2_quant_rows(x, group=128)
        # scales that are powers of two: codes times scale are 8-bit numbers, exact in bf16
        zc = torch.randint(-127, 128, (m, n), dtype=torch.int8, device="cuda")
        zs = torch.full((m, -(-n // 128)), 2.0 ** -5, device="cuda")
        z = mc2.mc2_dequant_rows(zc, zs, group=128)
        for act_code in range(5):
            xv = mc2.mc2_dequant_rows(xc, xs, group=128, act=act_code)
            got = mc2.mc2_linear_act_grad_i8(dout, xc, xs, w, zc, zs, act=act_code, x_act=act_code, group_offsets=off,
                                             need_dbias=True)
            want = mc2.mc2_linear_act_grad(dout, xv, w, z, act=act_code, group_offsets=off, need_dbias=True)
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_against_differences(mc2):
    """dx, dw and dbias of the operator against differences of the forward formula in 64 bits at the codes' values."""
    m, k, n = 6, 24, 40
    for name in ACTS:
        w, b, dout = rand(42, n, k, std=k ** -0.5), rand(43, n), rand(44, m, n)
        xc, xs = mc2.mc2_quant_rows(rand(41, m, k).cuda(), group=128)
        x = ref.values(xc.cpu(), xs.cpu(), 128)
        z = x @ w.double().T + b.double()
        # z kept in 8 bits is a z of its own: the bias takes up the difference, which is then the point of expansion
        zc, zs = mc2.mc2_quant_rows(z.bfloat16().cuda(), group=128)
        zv = ref.values(zc.cpu(), zs.cpu(), 128)
        shift = zv - z
        if name == "relu":  # away from its corner
            dout = torch.where(zv.abs() < 0.05, torch.zeros_like(dout), dout)
        got = mc2.mc2_linear_act_grad_i8(dout.cuda(), xc, xs, w.cuda(), zc, zs, act=ACTS.index(name), need_dbias=True)

        def loss(xv, wv, bv):
            return (act(xv @ wv.T + bv + shift, name)[0] * dout.double()).sum()

        d, base = 1e-5, [x, w.double(), b.double()]
        for i, g in enumerate(got):
            v = rand(45 + i, *base[i].shape).double()
            hi, lo = list(base), list(base)
            hi[i], lo[i] = base[i] + d * v, base[i] - d * v
            num = (loss(*hi) - loss(*lo)) / (2 * d)
            # x, dz and the result are each rounded to 8 bits
            g = g.cpu().double()
            tol = (4 * U["bf16"] * (g.abs() + 2.0) * v.abs()).sum()
            assert abs(num - (g * v).sum()) <= tol, (name, i)


def test_only_what_is_wanted_and_no_rows(mc2):
    xc, xs = mc2.mc2_quant_rows(rand(51, 70, 96).cuda(), group=128)
    zc, zs = mc2.mc2_quant_rows(rand(54, 70, 80).cuda(), group=128)
    w, dout = rand(52, 80, 96).cuda(), rand(53, 70, 80).cuda()
    kw = dict(act=mc2.MC2_ACT_SILU)
    full = mc2.mc2_linear_act_grad_i8(dout, xc, xs, w, zc, zs, need_dbias=True, **kw)
    for wanted in ((True, False, False), (False, True, False), (False, False, True), (True, True, False)):
        got = mc2.mc2_linear_act_grad_i8(dout, xc, xs, w, zc, zs, need_dx=wanted[0], need_dw=wanted[1],
                                         need_dbias=wanted[2], **kw)
        for on, a, b in zip(wanted, got, full):
            assert (a is not None) == on
            if on:
                assert torch.equal(a, b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = mc2.mc2_linear_act_grad_i8(dout, xc, xs, w, zc, zs, need_dbias=True, stream=st, **kw)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, full))
    dw, db = torch.full_like(w, 7.0), torch.full((80,), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = mc2.mc2_linear_act_grad_i8(dout[:0], xc[:0], xs[:0], w, zc[:0], zs[:0], need_dbias=True, dw=dw, dbias=db,
                                            **kw)
    assert dx.shape == (0, 96) and torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_graph_replay(mc2):
    x, w, dout = rand(61, 200, 320).cuda(), rand(62, 264, 320, std=1 / 16).cuda(), rand(63, 200, 264).cuda()
    b = rand(64, 264).cuda()

    def step():
        _, z = mc2.mc2_linear_act(x, w, b, act=mc2.MC2_ACT_GELU, need_z=True)
        xc, xs = mc2.mc2_quant_rows(x, group=128)
        zc, zs = mc2.mc2_quant_rows(z, group=128)
        return mc2.mc2_linear_act_grad_i8(dout, xc, xs, w, zc, zs, act=mc2.MC2_ACT_GELU, need_dbias=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (65, 66, 67):
        x.copy_(rand(seed, 200, 320))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, step()):
            assert torch.equal(a, c)


def test_a_group_that_is_nan_says_so(mc2):
    """Values that come back as NaN have a NaN in their gradients under every activation, relu's included."""
    m, k, n = 5, 64, 256
    w, dout = rand(71, n, k).cuda(), rand(72, m, n).cuda()
    xc, xs = mc2.mc2_quant_rows(rand(73, m, k).cuda(), group=128)
    z = rand(74, m, n)
    z[2, 3] = float("nan")
    zc, zs = mc2.mc2_quant_rows(z.cuda(), group=128)
    for code in range(1, 5):
        dx, dw, db = mc2.mc2_linear_act_grad_i8(dout, xc, xs, w, zc, zs, act=code, need_dbias=True)
        assert torch.isnan(dx[2]).all() and torch.isfinite(dx[[0, 1, 3, 4]]).all(), code
        assert torch.isnan(dw[:128]).all() and torch.isfinite(dw[128:]).all(), code
        assert torch.isnan(db[:128]).all() and torch.isfinite(db[128:]).all(), code


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_pre_activation_of_minus_infinity(mc2, dtype):
    """Kept with keep_inf its slope and its activation are 0 and its neighbours' what they are without it: the
    gradients of the formula where its dz and its column of the second linear's input are cleared."""
    m, k, n = 40, 136, 264
    u = U[dtype]
    w1, w2 = rand(81, n, k, std=k ** -0.5, dtype=dtype), rand(82, k, n, std=n ** -0.5, dtype=dtype)
    x, dout, z = rand(83, m, k, dtype=dtype), rand(84, m, n, dtype=dtype), rand(85, m, n, std=1.5, dtype=dtype)
    zero = z.clone()
    z[3, 5], z[3, 130], z[20, 263], z[39, :128] = -float("inf"), -float("inf"), -float("inf"), -float("inf")
    low = torch.isinf(z)
    zero[low] = 0.0
    xc, xs = mc2.mc2_quant_rows(x.cuda(), group=128)
    zc, zs = mc2.mc2_quant_rows(z.cuda(), group=128, keep_inf=True)
    v = ref.values(*ref.codes(zero, 128), 128)
    for name in ACTS[1:]:
        a, slope = act(v, name)
        a[low], slope[low] = 0.0, 0.0
        code = ACTS.index(name)
        dx, dw, db = mc2.mc2_linear_act_grad_i8(dout.cuda(), xc, xs, w1.cuda(), zc, zs, act=code, need_dbias=True)
        dz, xv = dout.double() * slope, ref.values(xc.cpu(), xs.cpu(), 128)
        # dz and the input are rounded to 16 bits, their sums in fp32; a slope is within ACT_ERR (1 + |z|)^3
        ez = (ACT_ERR * (1 + v.abs()) ** 3 + 4 * EPS32) * dout.double().abs() + u * dz.abs() + TINY[dtype]
        ez[low] = 0.0
        r = dz @ w1.double()
        check(dx, r, rounded(r, dtype) + (1 + u) * (ez + n * EPS32 * dz.abs()) @ w1.double().abs(), name)
        r = dz.T @ xv
        check(dw, r, rounded(r, dtype) + (1 + u) * ((ez + m * EPS32 * dz.abs()).T @ xv.abs() * (1 + u) +
                                                    dz.abs().T @ (u * xv.abs() + TINY[dtype])), name)
        r = dz.sum(0)
        check(db, r, rounded(r, dtype) + (1 + u) * (ez + (m + 8) * EPS32 * dz.abs()).sum(0), name)
        d2 = rand(86, m, k, dtype=dtype)
        _, dw2, _ = mc2.mc2_linear_act_grad_i8(d2.cuda(), zc, zs, w2.cuda(), x_act=code, need_dx=False)
        r = d2.double().T @ a
        ea = ACT_ERR * (1 + v.abs()) + 1.13 * EPS32 * v.abs() + u * a.abs() + TINY[dtype]
        check(dw2, r, rounded(r, dtype) + (1 + u) * d2.double().abs().T @ (ea + (m + 4) * EPS32 * a.abs()), name)
