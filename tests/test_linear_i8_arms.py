"""Every kernel that the plan of mc2_linear_i8 can choose, by (dense or grouped, tile or few rows, K whole or in parts):
on the CPU that the sizes below still reach each of them, on the GPU their results.

Sizes have partial tiles at both edges, partial and whole groups of four columns, a partial last step of K; the 256 x 256
tiles, which run their steps in pairs, have an odd and an even number of steps.  The bounds are test_gpu_linear_i8.py's.
"""
import ctypes
import math
import random

import pytest
import torch

import comm_matmul_tensor_amd as mc2
from layer_ref import ACT_ERR, DT, EPS32, U, act, rounded
from test_linear_arms import TILES, inputs, near

lib = ctypes.CDLL(mc2.LIB_PATH)
I = ctypes.c_int64


def arm(m, k, n, groups):
    """(grouped, tile or wavefronts of the few-row product, K in parts)"""
    tile, splits = ctypes.c_int(), ctypes.c_int()
    assert lib.mc2_testing_linear_i8_plan(I(m), I(k), I(n), I(groups), ctypes.byref(tile), ctypes.byref(splits)) == 0
    name = TILES[tile.value] if tile.value >= 0 else f"few rows, {-tile.value}"
    return groups > 0, name, splits.value > 1


# (m, k, n, groups): the arm of that product
CASES = [
    (6007, 516, 1290, 0, "256x256", False), (2764, 393, 2972, 0, "256x256", False),
    (1466, 522, 5692, 0, "256x256", False), (8322, 386, 923, 0, "256x256", False),
    (607, 400, 6979, 0, "128x256", False), (594, 397, 7132, 0, "128x256", False),
    (8229, 411, 321, 0, "128x128", False), (5484, 395, 544, 0, "128x128", False),
    (193, 19242, 2849, 0, "128x128", True), (106, 18182, 5468, 0, "128x128", True),
    (8472, 545, 193, 0, "96x128", False), (8570, 548, 220, 0, "96x128", False),
    (146, 13146, 2707, 0, "96x128", True), (140, 13216, 2848, 0, "96x128", True),
    (103, 397, 8243, 0, "128x64", False), (8697, 402, 144, 0, "128x64", False),
    (3199, 11906, 65, 0, "128x64", True), (4401, 10953, 68, 0, "128x64", True),
    (8394, 392, 67, 0, "96x64", False), (8931, 385, 68, 0, "96x64", False),
    (4440, 7380, 30, 0, "96x64", True), (2135, 7006, 72, 0, "96x64", True),
    (36, 422, 33, 0, "64x64", False), (40, 432, 32, 0, "64x64", False),
    (44, 3029, 31, 0, "64x64", True), (33, 3409, 32, 0, "64x64", True),
    (2, 401, 31, 0, "few rows, 16", False), (2, 406, 32, 0, "few rows, 16", False),
    (17, 1003, 2049, 0, "few rows, 16", False), (2, 394, 4287, 0, "few rows, 4", False),
    (1, 420, 4256, 0, "few rows, 4", False), (13, 1600, 4400, 0, "few rows, 4", False),
    (27, 407, 4289, 0, "few rows, 4", False), (32, 512, 4288, 0, "few rows, 4", False),
    (4298, 408, 1633, 13, "256x256", False), (1406, 550, 4750, 5, "256x256", False),
    (4438, 441, 1540, 13, "256x256", False), (1333, 527, 5144, 5, "256x256", False),
    (1739, 408, 1987, 13, "128x256", False), (5736, 387, 724, 13, "128x256", False),
    (998, 390, 2849, 3, "128x128", False), (6865, 392, 404, 13, "128x128", False),
    (6618, 522, 267, 5, "96x128", False), (1704, 531, 1092, 5, "96x128", False),
    (8164, 395, 70, 5, "96x64", False), (8136, 489, 76, 5, "96x64", False),
    (33, 391, 30, 3, "64x64", False), (35, 418, 32, 3, "64x64", False),
]


def test_sizes_reach_the_arms_they_name():
    for m, k, n, groups, name, parts in CASES:
        assert arm(m, k, n, groups) == (groups > 0, name, parts), (m, k, n, groups)


def test_every_arm_of_the_plan_is_named():
    """Arms over sizes of all orders: none but those above."""
    rng = random.Random(1)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    named = {(c[3] > 0, c[4], c[5]) for c in CASES}
    found = set()
    for _ in range(60000):
        found.add(arm(log(1, 70000), log(1, 100000), log(1, 30000), rng.choice([0, 0, 1, 2, 3, 5, 8, 13, 32, 300])))
    assert found <= named, found - named
    assert len(found) == len(named)


def test_few_rows_or_tiles():
    """Up to 8 rows always the few-row product; up to 32 while a CU's reads of x do not outweigh a tile's time."""
    for m, k, n, few in [(8, 16384, 28672, True), (16, 4096, 4096, True), (16, 4096, 28672, False), (16, 16384, 1024, False),
                         (32, 1024, 4096, True), (32, 8192, 8192, False), (33, 64, 64, False), (32, 512, 512, True)]:
        assert arm(m, k, n, 0)[1].startswith("few rows") == few, (m, k, n)
    for m, k, n, waves in [(1, 4096, 4096, 16), (1, 4096, 4097, 4), (1, 16384, 8192, 16), (1, 8192, 8192, 4)]:
        assert arm(m, k, n, 0)[1] == f"few rows, {waves}", (m, k, n)


# The tiles' cases with rows of a multiple of 4 bytes, not of 16: the last 4, 8 or 12 codes by themselves.
TAILS = [(m, k // 16 * 16 + 4 + 4 * (i % 3), n, groups, name, parts)
         for i, (m, k, n, groups, name, parts) in enumerate(CASES) if "rows" not in name]


def space(m, k, n, groups):
    got = ctypes.c_size_t()
    assert lib.mc2_linear_i8_workspace_size(I(m), I(k), I(n), I(groups), ctypes.byref(got)) == 0
    return got.value


def test_rows_read_where_they_stand():
    """Copied: rows of no multiple of 4, and of the others those of products that the copy makes faster."""
    for m, k, n, groups, name, parts in TAILS:
        assert arm(m, k, n, groups) == (groups > 0, name, parts), (m, k, n, groups)
    copied = [space(m, k, n, groups) >= (m + max(groups, 1) * n) * k for m, k, n, groups, _, _ in TAILS]
    assert copied.count(False) >= len(TAILS) - 4
    for m, k, n, groups, rows in [(4095, 4008, 5000, 0, True), (8191, 1000, 1000, 0, False), (64, 4008, 2040, 32, False),
                                  (64, 4006, 2040, 32, True), (64, 4096, 2040, 32, False), (517, 1001, 2000, 0, True)]:
        assert (space(m, k, n, groups) >= (m + max(groups, 1) * n) * k) == rows, (m, k, n, groups)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES + TAILS, ids=lambda c: "-".join(map(str, c)))
def test_results(case, dtype):
    m, k, n, groups = case[:4]
    rnd, lead, G, off, parts = inputs(m, k, n, groups, dtype)
    gen = torch.Generator(device="cuda").manual_seed(m)
    code = lambda *s: torch.randint(-128, 128, s, generator=gen, device="cuda", dtype=torch.int8)
    x, w, b, r = code(m, k), code(*lead, n, k), rnd(*lead, n, std=0.5), rnd(m, n)
    xs = torch.rand((m,), generator=gen, device="cuda") * 0.02 + 1e-3
    ws = (torch.rand((*lead, n), generator=gen, device="cuda") + 0.5) * (0.02 * k ** -0.5)
    out = mc2.mc2_linear_i8(x, xs, w, ws, b, r, act=mc2.MC2_ACT_SILU, group_offsets=off)
    z = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    ez = torch.zeros_like(z)
    for g, lo, hi in parts:
        p = (x[lo:hi].double() @ w.view(G, n, k)[g].double().t()) * xs[lo:hi, None].double() * ws.view(G, n)[g].double()
        z[lo:hi] = p + b.view(G, n)[g].double()
        ez[lo:hi] = 4 * EPS32 * (p.abs() + b.view(G, n)[g].double().abs())
    y = act(z, "silu")[0]
    want = y + r.double()
    bound = 1.13 * ez + ACT_ERR * (1 + z.abs()) + EPS32 * (y.abs() + r.double().abs())
    near(out, want, rounded(want, dtype) * (1 + U[dtype]) + bound, "out")


def test_rows_of_whole_chunks_are_never_copied():
    """Widths of a multiple of 16 bytes, whole cache lines or not, and widths of no multiple of 4 for comparison."""
    for m, n, groups in ((4096, 5000, 0), (4095, 1000, 0), (8192, 8192, 0), (8191, 1792, 32), (64, 2048, 32)):
        for k in (1008, 4000, 4080, 4096, 8176):
            assert space(m, k, n, groups) < (m + max(groups, 1) * n) * k, (m, k, n, groups)
            assert space(m, k + 1, n, groups) >= (m + max(groups, 1) * n) * k, (m, k + 1, n, groups)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(1000, 4000, 1000, 0), (4096, 4000, 640, 0), (33, 4080, 200, 0), (700, 4000, 264, 5),
                                  (2000, 1008, 520, 3)], ids=lambda c: "-".join(map(str, c)))
def test_results_of_widths_across_the_lines(case):
    test_results((*case, "", 1), "bf16")
