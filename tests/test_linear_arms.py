"""Every kernel that the plan of mc2_linear_act and mc2_linear_act_grad can choose, by (product, dense or grouped,
tile, K whole or in parts): on the CPU that the sizes below still reach each of them, on the GPU their results.

Sizes have partial tiles at both edges and a partial last step of K; the 256 x 256 tiles, which run their steps in
pairs, have an odd and an even number of steps.  The bounds are those of test_gpu_linear_act.py, taken on the GPU.
"""
import ctypes
import math
import random

import pytest
import torch

import comm_matmul_tensor_amd as mc2
from layer_ref import ACT_ERR, DT, EPS32, U, act, rounded, spans

lib = ctypes.CDLL(mc2.LIB_PATH)
I = ctypes.c_int64
FWD, DX, DW = 0, 1, 2
TILES = ["256x256", "128x256", "128x128", "96x128", "128x64", "96x64", "64x64"]


def arm(product, m, k, n, groups):
    """(product, grouped, tile or wavefronts of the few-row product, K in parts)"""
    tile, splits = ctypes.c_int(), ctypes.c_int()
    assert lib.mc2_testing_linear_plan(product, I(m), I(k), I(n), I(groups), ctypes.byref(tile), ctypes.byref(splits)) == 0
    name = TILES[tile.value] if tile.value >= 0 else f"few rows, {-tile.value}"
    return product, groups > 0, name, splits.value > 1


# (m, k, n, groups): the arm of that product
CASES = {
    FWD: [
        (8226, 329, 1092, 0, "256x256", False), (7366, 259, 1218, 0, "256x256", False),
        (487, 264, 8601, 0, "128x256", False), (292, 273, 8498, 0, "128x128", False),
        (8361, 326, 193, 0, "96x128", False), (97, 276, 8252, 0, "128x64", False), (67, 259, 8269, 0, "96x64", False),
        (35, 264, 33, 0, "64x64", False),
        (6216, 7617, 68, 0, "128x128", True), (4557, 5400, 66, 0, "96x128", True), (6146, 5994, 35, 0, "128x64", True),
        (1361, 3577, 67, 0, "96x64", True), (194, 2829, 155, 0, "64x64", True),
        (1550, 323, 4320, 13, "256x256", False), (1366, 265, 4813, 13, "256x256", False),
        (470, 258, 4729, 13, "128x256", False), (259, 265, 6297, 5, "128x128", False),
        (166, 329, 6443, 5, "96x128", False), (168, 266, 3186, 5, "96x64", False), (34, 263, 33, 3, "64x64", False),
        (1, 520, 7175, 0, "few rows, 4", False), (17, 1003, 7168, 0, "few rows, 4", False),
        (32, 4096, 6161, 0, "few rows, 4", False), (16, 77, 8009, 0, "few rows, 4", False),
        (1, 2051, 4090, 0, "few rows, 16", False), (17, 520, 2049, 0, "few rows, 16", False),
        (32, 1000, 4096, 0, "few rows, 16", False),
    ],
    DX: [
        (1744, 5201, 323, 0, "256x256", False), (2042, 4477, 262, 0, "256x256", False),
        (502, 8323, 260, 0, "128x256", False), (289, 8473, 258, 0, "128x128", False),
        (8600, 194, 326, 0, "96x128", False), (99, 8656, 264, 0, "128x64", False), (8351, 67, 266, 0, "96x64", False),
        (33, 33, 263, 0, "64x64", False),
        (6360, 65, 7677, 0, "128x128", True), (4165, 67, 5396, 0, "96x128", True), (3192, 67, 5965, 0, "128x64", True),
        (2740, 33, 3540, 0, "96x64", True), (654, 46, 2838, 0, "64x64", True),
        (1387, 4838, 324, 13, "256x256", False), (1441, 4557, 259, 13, "256x256", False),
        (514, 4552, 258, 13, "128x256", False), (673, 2426, 261, 13, "128x128", False),
        (164, 6473, 337, 5, "96x128", False), (7983, 66, 258, 13, "96x64", False), (33, 33, 270, 13, "64x64", False),
    ],
    DW: [
        (322, 966, 8258, 0, "256x256", False), (258, 8208, 927, 0, "256x256", False),
        (266, 6601, 579, 0, "128x256", False), (280, 8223, 195, 0, "128x128", False),
        (259, 8603, 66, 0, "128x64", False), (272, 33, 33, 0, "64x64", False),
        (7904, 4225, 66, 0, "128x128", True), (4346, 2699, 66, 0, "128x64", True), (2825, 43, 700, 0, "64x64", True),
        (4966, 129, 2444, 13, "256x256", False), (4159, 129, 2441, 13, "256x256", False),
        (4147, 2479, 33, 13, "128x256", False), (924, 35, 33, 3, "128x128", False),
    ],
}


def test_sizes_reach_the_arms_they_name():
    for product, cases in CASES.items():
        for m, k, n, groups, name, parts in cases:
            assert arm(product, m, k, n, groups) == (product, groups > 0, name, parts), (product, m, k, n, groups)


def test_every_arm_of_the_plan_is_named():
    """Arms over sizes of all orders: none but those above."""
    rng = random.Random(1)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    named = {(p, c[3] > 0, c[4], c[5]) for p, cases in CASES.items() for c in cases}
    found = set()
    for _ in range(40000):
        m, k, n, groups = log(1, 70000), log(1, 9000), log(1, 30000), rng.choice([0, 0, 1, 2, 3, 5, 8, 13, 32, 300])
        for p in (FWD, DX, DW):
            found.add(arm(p, m, k, n, groups))
    assert found <= named, found - named
    assert len(found) > 40


def test_few_rows_wavefronts():
    """16 wavefronts up to one workgroup (16 columns) per CU, and for 16 rows at most of a long K from two on; else 4."""
    for m, k, n, waves in [(1, 4096, 4096, 16), (1, 4096, 4097, 4), (32, 16384, 4096, 16), (32, 256, 4097, 4),
                           (16, 2048, 8192, 4), (16, 2048, 8193, 16), (17, 2048, 8193, 4), (16, 2047, 8193, 4),
                           (1, 1024, 28672, 4), (1, 8192, 28672, 16)]:
        assert arm(FWD, m, k, n, 0)[2] == f"few rows, {waves}", (m, k, n)


def test_plan_hook_refuses():
    t = ctypes.c_int()
    assert lib.mc2_testing_linear_plan(3, I(1), I(1), I(1), I(0), ctypes.byref(t), ctypes.byref(t)) == 4
    assert lib.mc2_testing_linear_plan(0, I(1), I(1), I(1), I(0), None, ctypes.byref(t)) == 1
    assert lib.mc2_testing_linear_plan(0, I(-1), I(1), I(1), I(0), ctypes.byref(t), ctypes.byref(t)) == 2


# ------------------------------------------------------------------ on the GPU
def near(got, ref, bound, what):
    assert got.shape == ref.shape
    bad = ~((got.double() - ref).abs() <= bound)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.numel()} outside the bound; first at {i}: got "
                             f"{got[i].item()!r} ref {ref[i].item()!r} bound {bound[i].item()!r}")


def ranges(m, groups):
    """Uneven ranges of rows: one empty, one of a single row, the last rows in none."""
    g = torch.Generator().manual_seed(groups)
    part = torch.rand((groups,), generator=g) + 0.3
    part[1] = 0.0
    end = (part.cumsum(0) / part.sum() * (m - max(1, m // 50))).long().tolist()
    end[0] = 1
    end[1] = 1
    return [0] + end


def inputs(m, k, n, groups, dtype):
    gen = torch.Generator(device="cuda").manual_seed(m + k + n)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(DT[dtype])
    G = max(groups, 1)
    lead = (groups,) if groups else ()
    offsets = ranges(m, groups) if groups else None
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    return rnd, lead, G, off, [(0, 0, m)] if offsets is None else spans(offsets, m)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES[FWD], ids=lambda c: "-".join(map(str, c)))
def test_forward(case, dtype):
    m, k, n, groups = case[:4]
    rnd, lead, G, off, parts = inputs(m, k, n, groups, dtype)
    x, w, b, r = rnd(m, k), rnd(*lead, n, k, std=1.5 * k ** -0.5), rnd(*lead, n, std=0.5), rnd(m, n)
    out, z = mc2.mc2_linear_act(x, w, b, r, act=mc2.MC2_ACT_SILU, group_offsets=off, need_z=True)
    ref = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(ref)
    for g, a, e in parts:
        wg, bg = w.view(G, n, k)[g].double(), b.view(G, n)[g].double()
        ref[a:e] = x[a:e].double() @ wg.t() + bg
        size[a:e] = x[a:e].double().abs() @ wg.t().abs() + bg.abs()
    ez = (k + 4) * EPS32 * size
    near(z, ref, rounded(ref, dtype) * (1 + U[dtype]) + ez, "z")
    y = act(ref, "silu")[0]
    want = y + r.double()
    bound = 1.13 * ez + ACT_ERR * (1 + ref.abs()) + EPS32 * (y.abs() + r.double().abs())
    near(out, want, rounded(want, dtype) * (1 + U[dtype]) + bound, "out")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES[DX] + CASES[DW], ids=lambda c: "-".join(map(str, c)))
def test_gradient(case, dtype):
    m, k, n, groups = case[:4]
    rnd, lead, G, off, parts = inputs(m, k, n, groups, dtype)
    x, dout, z, w = rnd(m, k), rnd(m, n), rnd(m, n, std=1.5), rnd(*lead, n, k, std=n ** -0.5)
    dx, dw, db = mc2.mc2_linear_act_grad(dout, x, w, z, act=mc2.MC2_ACT_SILU, group_offsets=off, need_dbias=True)
    u = U[dtype]
    zd = z.double()
    dz = dout.double() * act(zd, "silu")[1]
    ez = ACT_ERR * dout.double().abs() * (1 + zd.abs()) ** 3 + 2 * EPS32 * dz.abs()
    e16 = ez + u * dz.abs() + 2.0 ** -25  # dz as the products read it: its own error and its rounding
    rx = torch.zeros((m, k), dtype=torch.float64, device="cuda")
    sx = torch.zeros_like(rx)
    for g, a, e in parts:
        wg, xa, d = w.view(G, n, k)[g].double(), x[a:e].double(), dz[a:e]
        rx[a:e] = d @ wg
        sx[a:e] = e16[a:e] @ wg.abs() + (n + 4) * EPS32 * (d.abs() * (1 + u)) @ wg.abs()
        rw = d.t() @ xa
        sw = e16[a:e].t() @ xa.abs() + (e - a + 4) * EPS32 * (d.abs() * (1 + u)).t() @ xa.abs()
        near(dw.view(G, n, k)[g], rw, rounded(rw, dtype) * (1 + u) + sw, f"dw {g}")
        rb = d.sum(0)
        sb = ez[a:e].sum(0) + (e - a + 8) * EPS32 * d.abs().sum(0)
        near(db.view(G, n)[g], rb, rounded(rb, dtype) * (1 + u) + sb, f"dbias {g}")
    near(dx, rx, rounded(rx, dtype) * (1 + u) + sx, "dx")
