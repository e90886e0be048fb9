"""mc2_linear_i8 against its formula: exact integer sums, fp32 roundings after them (bound below), one of the output.

z = (c s) t + bias rounds at most four times in fp32: c to fp32, two products, the sum; 4 EPS32 (|c s t| + |bias|).
"""
import math

import pytest
import torch

from layer_ref import ACT_ERR, ACTS, DT, EPS32, U, act, check, rand, rounded, spans

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


def operands(seed, m, k, n, dtype, bias, residual, offsets, full=False):
    g = torch.Generator().manual_seed(seed)
    G = 0 if offsets is None else len(offsets) - 1
    lo = -128 if full else -127
    x = torch.randint(lo, 128, (m, k), generator=g, dtype=torch.int8)
    w = torch.randint(lo, 128, (G, n, k) if G else (n, k), generator=g, dtype=torch.int8)
    xs = torch.rand((m,), generator=g) * 0.02 + 1e-3
    ws = (torch.rand((G, n) if G else (n,), generator=g) + 0.5) * (0.02 * k ** -0.5)
    b = rand(seed + 2, *((G, n) if G else (n,)), std=0.5, dtype=dtype) if bias else None
    r = rand(seed + 3, m, n, dtype=dtype) if residual else None
    return x, xs, w, ws, b, r


def formula(x, xs, w, ws, b, r, name, groups):
    """(out, bound before the last rounding)"""
    m = x.shape[0]
    n = w.shape[-2]
    z, ez = torch.zeros((m, n), dtype=torch.float64), torch.zeros((m, n), dtype=torch.float64)
    for g, lo, hi in groups or [(None, 0, m)]:
        wg, wsg = (w, ws) if g is None else (w[g], ws[g])
        # (fp64 holds the sums of these products exactly)
        p = (x[lo:hi].double() @ wg.double().T) * xs[lo:hi, None].double() * wsg[None].double()
        bg = torch.zeros((n,), dtype=torch.float64) if b is None else (b if g is None else b[g]).double()
        z[lo:hi] = p + bg
        ez[lo:hi] = 4 * EPS32 * (p.abs() + bg.abs())
    out, _ = act(z, name)
    eo = 1.13 * ez + (0 if name in ("none", "relu") else ACT_ERR * (1 + z.abs()))
    if r is not None:
        eo = eo + EPS32 * (out.abs() + r.double().abs())
        out = out + r.double()
    return out, eo


def dev(t):
    return None if t is None else t.cuda()


def run(mc2, seed, m, k, n, dtype, name, bias, residual, offsets=None, full=False):
    x, xs, w, ws, b, r = operands(seed, m, k, n, dtype, bias, residual, offsets, full)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    out = mc2.mc2_linear_i8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), dev(b), dev(r), dtype=DT[dtype],
                            act=ACTS.index(name), group_offsets=off)
    ref, eo = formula(x, xs, w, ws, b, r, name, None if offsets is None else spans(offsets, m))
    assert out.dtype == DT[dtype]
    check(out, ref, rounded(ref, dtype) * (1 + U[dtype]) + eo, "out")


# few rows (one fragment or two), one tile and several, ragged everywhere, one of everything
SIZES = [(1, 1, 1), (1, 16, 16), (1, 4096, 1792), (2, 33, 7), (5, 264, 100), (16, 512, 4100), (17, 1000, 65),
         (32, 2049, 33), (33, 64, 64), (33, 63, 65), (64, 4096, 256), (100, 40, 1000), (129, 136, 127), (128, 16, 8),
         (257, 129, 131), (300, 200, 520), (517, 1792, 384), (1, 5, 3000), (256, 1, 256), (700, 72, 1), (1000, 576, 777),
         (9, 15, 40), (40, 4, 40), (40, 8, 41), (70, 12, 39), (100, 20, 64), (65, 1016, 100), (40, 15, 40), (40, 17, 41), (64, 128, 64), (64, 144, 64), (48, 31, 16)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sizes(mc2, m, k, n, dtype):
    print(f"linear_i8 m={m} k={k} n={n} {dtype}", flush=True)
    run(mc2, m + k + n, m, k, n, dtype, "gelu", True, True)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [3, 40, 200])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_epilogues(mc2, name, dtype, m, bias, residual):
    run(mc2, 11, m, 336, 296, dtype, name, bias, residual)


@pytest.mark.parametrize("m,k,n", [(4096, 512, 4096), (2048, 640, 2048), (4100, 400, 3850), (512, 1024, 4096),
                                   (381, 300, 4090), (509, 150, 4091), (761, 912, 4088), (250, 272, 4088), (70, 4112, 1030)])
def test_larger_tiles(mc2, m, k, n):
    print(f"linear_i8 m={m} k={k} n={n}", flush=True)
    run(mc2, 5, m, k, n, "bf16", "silu", True, True)


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
    (1, [0, 0, 1]),
]


@pytest.mark.parametrize("m,offsets", GROUPS)
@pytest.mark.parametrize("k,n", [(512, 128), (400, 264), (77, 39), (4, 39), (204, 264), (136, 40), (76, 39)])
def test_groups(mc2, m, offsets, k, n):
    print(f"groups m={m} k={k} n={n} offsets={offsets[:8]}", flush=True)
    run(mc2, 21, m, k, n, "bf16", "silu", True, True, offsets)
    run(mc2, 22, m, k, n, "f16", "none", False, False, offsets)


def many_groups(m, groups):
    """Ranges of 0 to 60 rows, every fifth one empty, one end out of order, rows left over."""
    g = torch.Generator().manual_seed(groups)
    sizes = torch.randint(0, 61, (groups,), generator=g)
    sizes[::5] = 0
    offsets = [0] + (sizes.cumsum(0) * (m - 9) // sizes.sum()).tolist()
    offsets[groups // 2] = offsets[groups // 3]
    return offsets


def test_many_groups(mc2):
    run(mc2, 24, 3000, 144, 136, "bf16", "silu", True, True, many_groups(3000, 700))
    run(mc2, 25, 9000, 64, 520, "f16", "none", True, False, many_groups(9000, 129))
    run(mc2, 26, 200, 300, 1100, "f16", "gelu", True, True, many_groups(200, 90))


def test_groups_large_tiles(mc2):
    run(mc2, 23, 2500, 384, 2048, "bf16", "gelu", True, False, [0, 700, 1500, 1501, 2470])


@pytest.mark.parametrize("m", [1, 20, 40, 300])
def test_the_longest_sums(mc2, m):
    """k of 2^17 - 1 with all codes at their ends: the largest sums that int32 holds."""
    k, n = (1 << 17) - 1, 40
    xs, ws = torch.full((m,), 1e-4), torch.full((n,), 1e-4)
    for a, b in ((-128, -128), (127, 127), (-128, 127)):
        x, w = torch.full((m, k), a, dtype=torch.int8), torch.full((n, k), b, dtype=torch.int8)
        out = mc2.mc2_linear_i8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), dtype=torch.bfloat16)
        want = torch.full((m, n), float(a * b * k) * float(xs[0]) * float(ws[0]), dtype=torch.float64)
        check(out, want, rounded(want, "bf16") + 4 * EPS32 * want.abs(), "out")


def test_scales_as_the_quantisers_give_them(mc2):
    """The whole chain: a norm's codes and a weight's by channel; scales of one column."""
    x, wn = rand(41, 37, 256).cuda(), rand(42, 256).cuda()
    w = rand(43, 72, 256, std=1 / 16).cuda()
    q, qs, _, _ = mc2.mc2_add_rms_norm(x, wn, out_dtype=torch.int8)
    wq, wqs = mc2.mc2_quant_rows(w)
    assert qs.shape == (37, 1) and wqs.shape == (72, 1)
    a = mc2.mc2_linear_i8(q, qs, wq, wqs)
    b = mc2.mc2_linear_i8(q, qs.view(-1), wq, wqs.view(-1), dtype=torch.bfloat16)
    assert torch.equal(a, b) and a.dtype == torch.bfloat16
    full, _ = mc2.mc2_linear_act(mc2.mc2_add_rms_norm(x, wn)[0], w)
    # 8 bits against 16: each factor off by half a step of 1 / 127 of its row's largest value at most
    xf = q.cpu().double() * qs.cpu().double()
    wf = wq.cpu().double() * wqs.cpu().double()
    slack = 0.5 * (qs.cpu().double() @ wf.abs().sum(1)[None] + xf.abs().sum(1)[:, None] @ wqs.cpu().double().T) * 1.02
    check(a, full.cpu().double(), slack + 4 * U["bf16"] * full.cpu().double().abs() + 1e-3, "8 bits against 16")
    w3 = rand(44, 3, 72, 256, std=1 / 16).cuda()
    w3q, w3s = mc2.mc2_quant_rows(w3)
    off = torch.tensor([0, 10, 10, 30], dtype=torch.int32).cuda()
    c = mc2.mc2_linear_i8(q, qs, w3q, w3s, group_offsets=off)
    assert torch.equal(c[:10], mc2.mc2_linear_i8(q[:10].contiguous(), qs[:10].contiguous(), w3q[0], w3s[0]))
    assert torch.count_nonzero(c[30:]) == 0


def test_odd_scales(mc2):
    """Scales of 0, NaN and infinity stay in their rows and columns; rows of no group are 0 whatever theirs are."""
    for m, offsets in ((8, None), (24, None), (200, None), (200, [0, 90, 150])):
        x, xs, w, ws, _, _ = operands(61, m, 144, 72, "bf16", False, False, offsets)
        off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
        clean = mc2.mc2_linear_i8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), group_offsets=off).cpu()
        bad = xs.clone()
        bad[0], bad[3], bad[m - 1] = 0.0, math.nan, math.inf
        got = mc2.mc2_linear_i8(x.cuda(), bad.cuda(), w.cuda(), ws.cuda(), group_offsets=off).cpu()
        others = [i for i in range(m) if i not in (0, 3, m - 1)]
        assert torch.equal(got[others], clean[others])
        assert torch.count_nonzero(got[0]) == 0 and torch.isnan(got[3]).all()
        if offsets is None:
            assert not torch.isfinite(got[m - 1].float()).any()
        else:
            assert torch.count_nonzero(got[150:]) == 0
        wbad = ws.clone()
        wbad[..., 71] = math.nan
        got = mc2.mc2_linear_i8(x.cuda(), xs.cuda(), w.cuda(), wbad.cuda(), group_offsets=off).cpu()
        assert torch.equal(got[:, :71], clean[:, :71])
        end = 150 if offsets else m
        assert torch.isnan(got[:end, 71]).all() and torch.count_nonzero(got[end:]) == 0


def test_residual_in_place_streams_and_no_rows(mc2):
    for m, offsets in ((5, None), (150, None), (400, None), (700, [0, 300, 300, 650])):
        x, xs, w, ws, b, r = operands(58, m, 320, 264, "bf16", True, True, offsets)
        off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
        args = (x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), b.cuda())
        r = r.cuda()
        want = mc2.mc2_linear_i8(*args, r, act=mc2.MC2_ACT_GELU, group_offsets=off)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        other = mc2.mc2_linear_i8(*args, r, act=mc2.MC2_ACT_GELU, group_offsets=off, stream=st)
        st.synchronize()
        assert torch.equal(want, other)
        got = mc2.mc2_linear_i8(*args, r, act=mc2.MC2_ACT_GELU, group_offsets=off, out=r)
        assert got is r and torch.equal(got, want)
    out = mc2.mc2_linear_i8(x[:0].cuda(), xs[:0].cuda(), w[0].cuda(), ws[0].cuda(), b[0].cuda())
    assert out.shape == (0, 264)
    out = mc2.mc2_linear_i8(x[:0].cuda(), xs[:0].cuda(), w.cuda(), ws.cuda(), group_offsets=off)
    assert out.shape == (0, 264)


def test_nothing_outside_is_written(mc2):
    for m, k, n, offsets in ((3, 100, 33, None), (50, 100, 33, None), (50, 128, 72, [0, 20, 45])):
        x, xs, w, ws, _, _ = operands(59, m, k, n, "bf16", False, False, offsets)
        off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
        buf = torch.full((m + 4, n), 7.0, dtype=torch.bfloat16, device="cuda")
        mc2.mc2_linear_i8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), group_offsets=off, out=buf[:m])
        assert (buf[m:] == 7.0).all()


def test_offsets_past_32_bits(mc2):
    """Operands of more than 2^31 codes: the last rows and columns of the result."""
    k, n = 65536, 33000
    w = torch.zeros((n, k), dtype=torch.int8, device="cuda")
    g = torch.Generator().manual_seed(3)
    tail = torch.randint(-127, 128, (8, k), generator=g, dtype=torch.int8)
    w[-8:] = tail.cuda()
    ws = torch.full((n,), 1e-3)
    for m in (2, 48):
        x = torch.randint(-127, 128, (m, k), generator=g, dtype=torch.int8)
        xs = torch.rand((m,), generator=g)
        out = mc2.mc2_linear_i8(x.cuda(), xs.cuda(), w, ws.cuda())
        want = (x.double() @ tail.double().T) * xs.double()[:, None] * ws.double()[0]
        check(out[:, -8:], want, rounded(want, "bf16") + 4 * EPS32 * want.abs(), "out")
        assert torch.count_nonzero(out[:, :8]) == 0
    w2 = torch.randint(-127, 128, (24, k), generator=g, dtype=torch.int8)
    ones = torch.ones((24,))
    out = mc2.mc2_linear_i8(w, ws.cuda(), w2.cuda(), ones.cuda())
    want = (tail.double() @ w2.double().T) * ws.double()[0]
    check(out[-8:], want, rounded(want, "bf16") + 4 * EPS32 * want.abs(), "out")
    off = torch.tensor([0, 100, n], dtype=torch.int32).cuda()
    out = mc2.mc2_linear_i8(w, ws.cuda(), torch.stack([w2, w2]).cuda(), torch.stack([ones, ones]).cuda(), group_offsets=off)
    check(out[-8:], want, rounded(want, "bf16") + 4 * EPS32 * want.abs(), "out, grouped")


def test_graph_replay(mc2):
    """Codes of rows into the product of few rows, a split one and experts' products, captured and replayed."""
    src = rand(70, 96, 4096).cuda()
    w, ws = mc2.mc2_quant_rows(rand(71, 64, 4096, std=1 / 64).cuda())
    w3, ws3 = mc2.mc2_quant_rows(rand(72, 3, 40, 4096, std=1 / 64).cuda())
    off = torch.tensor([0, 30, 30, 90], dtype=torch.int32).cuda()

    def calls():
        q, s = mc2.mc2_quant_rows(src)
        return (mc2.mc2_linear_i8(q, s, w, ws, act=mc2.MC2_ACT_SILU),
                mc2.mc2_linear_i8(q[:7], s[:7], w, ws),
                mc2.mc2_linear_i8(q, s, w3, ws3, group_offsets=off))

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for seed in (73, 74, 75):
        src.copy_(rand(seed, 96, 4096))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, calls()):
            assert torch.equal(a, b)
