"""mc2_quant_rows: the codes and scales of its definition, bit for bit; mc2_dequant_rows: one rounding from theirs."""
import math

import pytest
import torch

import layer8_ref as ref
from layer_ref import ACT_ERR, ACTS, DT, EPS32, TINY, U, act, check, rand, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


def run(mc2, x, group, names=("none",), dtype="bf16"):
    codes, scale = mc2.mc2_quant_rows(x.cuda(), group=group)
    want, ws = ref.codes(x, group)
    assert codes.dtype == torch.int8 and scale.shape == ws.shape
    assert torch.equal(scale.cpu().view(torch.int32)[~torch.isnan(ws)], ws.view(torch.int32)[~torch.isnan(ws)])
    assert torch.equal(torch.isnan(scale.cpu()), torch.isnan(ws))
    assert torch.equal(codes.cpu(), want)
    for name in names:
        back = mc2.mc2_dequant_rows(codes, scale, group=group, act=ACTS.index(name), dtype=DT[dtype])
        v = ref.values(want, ws, group)
        y, slope = act(v, name)
        # the product code * scale rounds once in fp32 before the activation
        err = EPS32 * v.abs() * 1.13 + (0 if name in ("none", "relu") else ACT_ERR * (1 + v.abs()))
        check(back, y, rounded(y, dtype) + (1 + U[dtype]) * err, name)
    return codes, scale


SIZES = [(1, 1), (1, 7), (3, 8), (2, 127), (5, 128), (4, 129), (1, 512), (9, 513), (3, 1000), (2, 1024), (7, 1025),
         (3, 2047), (2, 4096), (3, 4100), (2, 7168), (2, 8193), (1, 16384), (2, 20001), (1, 32768), (2, 40000), (1, 65537),
         (300, 64), (257, 200), (1000, 33)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [0, 128])
def test_sizes(mc2, rows, cols, dtype, group):
    print(f"codes {rows} x {cols} {dtype} group {group}", flush=True)
    run(mc2, rand(rows + cols, rows, cols, std=3.0, dtype=dtype), group, dtype=dtype)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group,cols", [(0, 200), (128, 256), (128, 333)])
def test_activations(mc2, name, dtype, group, cols):
    run(mc2, rand(3, 40, cols, std=2.0, dtype=dtype), group, (name,), dtype)


@pytest.mark.parametrize("group", [0, 128])
def test_extremes(mc2, group):
    """Zeros, one value, the smallest and largest numbers, halves of a step, NaN and infinity in one group."""
    for dtype, tiny, huge in (("bf16", 2.0 ** -133, 3.38e38), ("f16", 2.0 ** -24, 65504.0)):
        x = torch.zeros((9, 300), dtype=torch.float64)
        x[1, 200] = 2.0
        x[2, :] = tiny
        x[3, ::3] = -huge
        x[4] = torch.linspace(-127, 127, 300)
        x[5] = (torch.arange(300) % 255 - 127) / 2  # halves of a step: ties to even
        x[5, 0] = x[5, 128] = x[5, 256] = 127
        x[6] = torch.linspace(-1e-3, 1e-3, 300)
        x[7] = 1.0
        x[8] = -x[4]
        run(mc2, x.to(DT[dtype]), group, dtype=dtype) if dtype == "f16" else run(mc2, x.to(DT[dtype]), group, (), dtype)
        y = rand(8, 4, 300, dtype=dtype)
        y[0, 5], y[1, 290], y[2, 7] = math.nan, math.inf, -math.inf
        codes, scale = mc2.mc2_quant_rows(y.cuda(), group=group)
        want, ws = ref.codes(torch.where(torch.isfinite(y), y, torch.zeros_like(y)), group)
        width = group or 300
        for row, col in ((0, 5), (1, 290), (2, 7)):
            g = col // width
            assert not math.isfinite(float(scale[row, g]))
            assert torch.count_nonzero(codes[row, g * width:(g + 1) * width]) == 0
            back = mc2.mc2_dequant_rows(codes, scale, group=group, dtype=DT[dtype])
            assert torch.isnan(back[row, g * width:(g + 1) * width]).all()
            ws[row, g] = float(scale[row, g])
            want[row, g * width:(g + 1) * width] = 0
        assert torch.equal(codes.cpu(), want)
        finite = torch.isfinite(ws)
        assert torch.equal(scale.cpu()[finite], ws[finite])


def test_shapes_outputs_given_and_streams(mc2):
    x = rand(4, 6, 5, 136).cuda()
    codes, scale = mc2.mc2_quant_rows(x, group=128)
    assert codes.shape == (6, 5, 136) and scale.shape == (6, 5, 2)
    flat = mc2.mc2_quant_rows(x.view(30, 136), group=128)
    assert torch.equal(flat[0].view_as(codes), codes) and torch.equal(flat[1].view_as(scale), scale)
    one = mc2.mc2_quant_rows(x[0, 0].contiguous())
    assert one[0].shape == (136,) and one[1].shape == (1,)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c2, s2 = torch.empty_like(codes), torch.empty_like(scale)
    got = mc2.mc2_quant_rows(x, group=128, codes=c2, scale=s2, stream=st)
    back = mc2.mc2_dequant_rows(c2, s2, group=128, out=torch.empty_like(x), stream=st)
    st.synchronize()
    assert got[0] is c2 and torch.equal(c2, codes) and torch.equal(s2, scale)
    assert torch.equal(back, mc2.mc2_dequant_rows(codes, scale, group=128))
    empty = torch.empty((0, 136), dtype=torch.bfloat16, device="cuda")
    codes, scale = mc2.mc2_quant_rows(empty)
    assert codes.shape == (0, 136) and scale.shape == (0, 1)
    assert mc2.mc2_dequant_rows(codes, scale).shape == (0, 136)


def test_nothing_outside_is_written(mc2):
    """Rows behind the last one, and bytes past a ragged row's end, stay as they were."""
    for cols in (128, 131, 4099):
        for group in (0, 128):
            x = rand(9, 3, cols).cuda()
            buf = torch.full((5, cols), 77, dtype=torch.int8, device="cuda")
            per = -(-cols // 128) if group else 1
            sc = torch.full((5, per), 7.0, device="cuda")
            mc2.mc2_quant_rows(x, group=group, codes=buf[:3], scale=sc[:3])
            assert (buf[3:] == 77).all() and (sc[3:] == 7.0).all()
            out = torch.full((5, cols), 7.0, dtype=torch.bfloat16, device="cuda")
            mc2.mc2_dequant_rows(buf[:3], sc[:3], group=group, out=out[:3])
            assert (out[3:] == 7.0).all()


def test_offsets_past_32_bits(mc2):
    rows, cols = 70000, 32776
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = rand(10, 4, cols)
    x[-4:] = tail.cuda()
    for group in (0, 128):
        codes, scale = mc2.mc2_quant_rows(x, group=group)
        want, ws = ref.codes(tail, group)
        assert torch.equal(codes[-4:].cpu(), want) and torch.equal(scale[-4:].cpu(), ws)
        assert torch.count_nonzero(codes[0]) == 0
        back = mc2.mc2_dequant_rows(codes, scale, group=group, out=x)
        v = ref.values(want, ws, group)
        check(back[-4:], v, rounded(v, "bf16") * 1.01, "back")
        x[-4:] = tail.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cols", [128, 300, 1024, 4099])
def test_infinities_that_are_kept(mc2, dtype, cols):
    """keep_inf: the scale is that of the finite values (the type's largest number where there are none but zeros), +inf
    takes its place at the end of the range, -inf comes back as one; finite groups are those of group 128 bit for bit,
    and a NaN still makes its group NaN."""
    big = 65504.0 if dtype == "f16" else torch.finfo(torch.bfloat16).max
    x = rand(cols, 12, cols, std=2.0, dtype=dtype)
    inf = math.inf
    x[1, 5] = -inf
    x[2, 5], x[2, 77], x[2, 127] = inf, inf, 0.0
    x[3, 5], x[3, 6] = -inf, inf
    x[4, :128] = -inf
    x[5, :128] = 0.0
    x[5, 17], x[5, 99] = -inf, inf
    x[6, :128] = inf
    x[7, 5], x[7, 6] = math.nan, -inf
    x[8, cols - 1] = -inf                      # the last group, which may be short
    x[9, ::2] = -inf
    x[10, :128] = -0.0
    codes, scale = mc2.mc2_quant_rows(x.cuda(), group=128, keep_inf=True)
    codes, scale = codes.cpu(), scale.cpu()
    plain = mc2.mc2_quant_rows(x.cuda(), group=128)
    back = {name: mc2.mc2_dequant_rows(codes.cuda(), scale.cuda(), group=128, act=ACTS.index(name), dtype=DT[dtype]).cpu()
            for name in ACTS}
    for r in range(12):
        for g in range(scale.shape[1]):
            at = slice(128 * g, min(128 * g + 128, cols))
            v, c, s = x[r, at].float(), codes[r, at], scale[r, g]
            if torch.isnan(v).any():
                assert torch.isnan(s) and torch.count_nonzero(c) == 0
                assert all(torch.isnan(b[r, at]).all() for b in back.values())
                continue
            low, lost = v == -inf, torch.isinf(v)
            if not lost.any():
                assert torch.equal(c, plain[0][r, at].cpu()) and s == plain[1][r, g].cpu()
                continue
            top = v[~lost].abs().max() if (~lost).any() else torch.zeros(())
            top = top if top > 0 else torch.tensor(big)
            want = -(top / 127) if low.any() else top / 127
            assert s == want, (r, g)
            q = torch.round(v.clamp(-float(top), float(top)) / want).to(torch.int8)
            q[low] = -128
            assert torch.equal(c, q), (r, g)
            assert (back["none"][r, at][low] == -inf).all()
            assert torch.equal(torch.isinf(back["none"][r, at]), low) or top == big
            for name in ACTS[1:]:
                assert (back[name][r, at][low] == 0).all() and not torch.isnan(back[name][r, at]).any(), name


def test_no_infinity_no_difference(mc2):
    for rows, cols in ((1, 1), (3, 131), (70, 2048), (2, 7168)):
        x = rand(rows + cols, rows, cols).cuda()
        for a, b in zip(mc2.mc2_quant_rows(x, group=128), mc2.mc2_quant_rows(x, group=128, keep_inf=True)):
            assert torch.equal(a, b)
