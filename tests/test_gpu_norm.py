"""mc2_add_rms_norm and its gradient against their formulas in 64 bits.

Bounds: fp32 statistics of h terms are within (h / 64 + 32) roundings of the
exact ones (64 lanes at least share a row), so y is within that, a few more
roundings and the output's own.  Codes: a value within that distance of a
rounding boundary may go either way, so a code's value is within half a step
plus the bound.
"""
import pytest
import torch

from layer_ref import DT, EPS32, TINY, U, check, norm, norm_grad, rand, rounded

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


def stat_err(h):
    return (h / 64 + 32) * EPS32


WIDTHS = [1, 7, 8, 64, 127, 512, 520, 1000, 1024, 2048, 2049, 4096, 5000, 7168, 8192, 8200, 16384, 20001, 32768, 40000]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("h", WIDTHS)
@pytest.mark.parametrize("residual", [True, False])
def test_norm(mc2, h, dtype, residual):
    rows = 3 if h > 4096 else 9
    print(f"norm h={h} {dtype} residual={residual}", flush=True)
    x, w = rand(1, rows, h, dtype=dtype), rand(3, h, dtype=dtype)
    r = rand(2, rows, h, std=3.0, dtype=dtype) if residual else None
    out, scale, s, rstd = mc2.mc2_add_rms_norm(x.cuda(), w.cuda(), None if r is None else r.cuda(), eps=EPS,
                                               need_rstd=True)
    ref_s, ref_rstd, y = norm(x, r, w, EPS)
    assert scale is None and out.dtype == DT[dtype]
    check(rstd, ref_rstd, stat_err(h) * ref_rstd, "rstd")
    check(out, y, rounded(y, dtype) + (stat_err(h) + 4 * EPS32) * 2 * y.abs(), "out")
    if residual:
        check(s, ref_s, rounded(ref_s, dtype) + EPS32 * ref_s.abs(), "sum")
    else:
        assert torch.equal(s.cpu(), x)


@pytest.mark.parametrize("rows", [0, 1, 2, 3, 5, 257, 1030])
def test_norm_rows(mc2, rows):
    x, r, w = rand(4, rows, 264), rand(5, rows, 264), rand(6, 264)
    out, _, s, rstd = mc2.mc2_add_rms_norm(x.cuda(), w.cuda(), r.cuda(), eps=EPS, need_rstd=True)
    ref_s, _, y = norm(x, r, w, EPS)
    check(out, y, rounded(y, "bf16") + 1e-5 * y.abs(), "out")
    check(s, ref_s, rounded(ref_s, "bf16"), "sum")
    if rows:
        dx, dw = mc2.mc2_add_rms_norm_grad(out, s, w.cuda(), rstd)
        ref_dx, ref_dw = norm_grad(out.cpu(), None, s.cpu(), w, rstd.cpu())
        assert dx.shape == (rows, 264)
        check(dw, ref_dw, rounded(ref_dw, "bf16") + (rows + 64) * EPS32 *
              (out.cpu().double() * s.cpu().double() * rstd.cpu().double()[:, None]).abs().sum(0), "dweight")
    else:
        dx, dw = mc2.mc2_add_rms_norm_grad(x.cuda(), x.cuda(), w.cuda(), rstd)
        assert dx.shape == (0, 264) and torch.equal(dw.cpu(), torch.zeros(264, dtype=torch.bfloat16))


@pytest.mark.parametrize("kind", ["i8", "f8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("h,group", [(1, 0), (13, 0), (128, 128), (640, 128), (1024, 0), (2048, 128), (4097, 0),
                                     (7168, 0), (7168, 128), (9000, 0), (32768, 128), (33024, 128), (33000, 0)])
def test_norm_codes(mc2, h, group, dtype, kind):
    print(f"codes h={h} group={group} {dtype} {kind}", flush=True)
    x, r, w = rand(7, 5, h, dtype=dtype), rand(8, 5, h, std=2.0, dtype=dtype), rand(9, h, dtype=dtype)
    out_dtype, top = (torch.int8, 127.0) if kind == "i8" else (torch.float8_e4m3fn, 448.0)
    q, scale, s, rstd = mc2.mc2_add_rms_norm(x.cuda(), w.cuda(), r.cuda(), eps=EPS, out_dtype=out_dtype, group=group,
                                             need_rstd=True)
    _, ref_rstd, y = norm(x, r, w, EPS)
    g = group or h
    ref_scale = y.view(5, -1, g).abs().amax(2) / top
    err = 2 * (stat_err(h) + 4 * EPS32)
    assert q.dtype == out_dtype and scale.shape == ref_scale.shape
    check(scale, ref_scale, (err + EPS32) * ref_scale, "scale")
    codes, sc = q.cpu().to(torch.float64).view(5, -1, g), scale.cpu().double()[:, :, None]
    assert codes.abs().max() <= top
    yg = y.view(5, -1, g)
    if kind == "i8":
        step = sc * torch.ones_like(yg)
    else:  # E4M3: 4 significand bits, spacing 2^-9 at the least
        t = (yg / sc).abs().clamp(min=2.0 ** -6)
        step = sc * 2.0 ** (torch.floor(torch.log2(t * (1 + 1e-4))) - 3)
    check((codes * sc).view(5, h), y, (0.5 * step + (err + 4 * EPS32) * yg.abs() + 1e-4 * step).view(5, h), "values")


def test_norm_codes_special_rows(mc2):
    """Rows of zeros, of one value, with an infinity, with a NaN and of subnormal size."""
    h = 512
    x = torch.zeros(6, h)
    x[1], x[2, 5], x[3, 7] = 2.0, float("inf"), float("nan")
    x[4] = torch.linspace(-1, 1, h)
    x[5, 100] = 1.0
    w = torch.ones(h)
    for out_dtype, top in ((torch.int8, 127.0), (torch.float8_e4m3fn, 448.0)):
        q, scale, _, _ = mc2.mc2_add_rms_norm(x.bfloat16().cuda(), w.bfloat16().cuda(), eps=EPS, out_dtype=out_dtype)
        q, scale = q.cpu().float(), scale.cpu()
        assert torch.all(q[0] == 0) and scale[0] == 0
        assert torch.all(q[1] == top)
        # an infinity makes rstd 0 and its own value NaN: the row's scale says so, its codes are 0
        assert torch.all(q[2] == 0) and not torch.isfinite(scale[2])
        assert torch.all(q[3] == 0) and torch.isnan(scale[3])
        assert q[4].min() == -top and q[4].max() == top
        assert q[5, 100] == top and torch.all(q[5, :100] == 0)
        q2, scale2, _, _ = mc2.mc2_add_rms_norm(x.bfloat16().cuda(), w.bfloat16().cuda(), eps=EPS, out_dtype=out_dtype,
                                                group=128)
        q2, scale2 = q2.cpu().float(), scale2.cpu()
        assert scale2[5, 1:].abs().max() == 0 and torch.all(q2[5, 128:] == 0) and q2[5, 100] == top
        assert torch.isnan(scale2[3]).all()  # rstd is the row's


def test_norm_int8_feeds_the_static_product(mc2):
    """Codes and per-token scales as mc2_alltoall_quant_matmul_static takes them: two ranks' halves of
    the columns, each normed and coded over its own half of the tokens' columns."""
    tokens, h, n = 48, 256, 64
    g = torch.Generator().manual_seed(3)
    w8 = torch.randint(-127, 128, (h, n), generator=g, dtype=torch.int8)
    x, w = rand(10, tokens, h), rand(11, h)
    q, scale, _, _ = mc2.mc2_add_rms_norm(x.cuda(), w.cuda(), eps=EPS, out_dtype=torch.int8)
    x1 = torch.cat([q[:, :h // 2], q[:, h // 2:]]).contiguous()  # block j: what rank j sent
    s2 = torch.full((n,), 1e-3, device="cuda")
    out = mc2.mc2_alltoall_quant_matmul_static(x1, 2, scale[:, 0].contiguous(), w8.cuda(), s2)
    want = (q.cpu().double() @ w8.double()) * scale.cpu().double() * 1e-3
    check(out, want, rounded(want, "bf16") + 1e-6 * want.abs() + 1e-9, "product")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("h", [1, 9, 64, 512, 1000, 1024, 2048, 4096, 4100, 8192, 16000, 32768, 33001])
@pytest.mark.parametrize("with_dsum", [True, False])
def test_norm_grad(mc2, h, dtype, with_dsum):
    rows = 4 if h > 8192 else 37
    print(f"norm_grad h={h} {dtype} dsum={with_dsum}", flush=True)
    s, dout, w = rand(12, rows, h, std=2.0, dtype=dtype), rand(13, rows, h, dtype=dtype), rand(14, h, dtype=dtype)
    dsum = rand(15, rows, h, dtype=dtype) if with_dsum else None
    rstd = (1 / torch.sqrt((s.double() ** 2).mean(1) + EPS)).float()
    dx, dw = mc2.mc2_add_rms_norm_grad(dout.cuda(), s.cuda(), w.cuda(), rstd.cuda(),
                                       None if dsum is None else dsum.cuda())
    ref_dx, ref_dw = norm_grad(dout, dsum, s, w, rstd)
    r = rstd.double()[:, None]
    g = (dout.double() * w.double()).abs()
    terms = r * (g + s.double().abs() * r * r * (g * s.double().abs()).mean(1, keepdim=True))
    if with_dsum:
        terms = terms + dsum.double().abs()
    check(dx, ref_dx, rounded(ref_dx, dtype) + (stat_err(h) + 8 * EPS32) * terms, "dx")
    size = (dout.double() * s.double() * r).abs().sum(0)
    check(dw, ref_dw, rounded(ref_dw, dtype) + (rows + 32) * EPS32 * size, "dweight")


def test_norm_grad_many_rows(mc2):
    """More rows than workgroups that walk them, and the partial sums of all of them."""
    rows, h = 5003, 192
    s, dout, w = rand(16, rows, h), rand(17, rows, h), rand(18, h)
    rstd = (1 / torch.sqrt((s.double() ** 2).mean(1) + EPS)).float()
    dx, dw = mc2.mc2_add_rms_norm_grad(dout.cuda(), s.cuda(), w.cuda(), rstd.cuda())
    ref_dx, ref_dw = norm_grad(dout, None, s, w, rstd)
    size = (dout.double() * s.double() * rstd.double()[:, None]).abs().sum(0)
    check(dw, ref_dw, rounded(ref_dw, "bf16") + 300 * EPS32 * size, "dweight")
    check(dx, ref_dx, rounded(ref_dx, "bf16") + 1e-4, "dx")


def test_norm_grad_differences(mc2):
    """dx and dweight against central differences of the forward formula in 64 bits."""
    rows, h = 3, 48
    x, r, w, dout, dsum = (rand(20 + i, *(rows, h) if i != 2 else (h,)) for i in range(5))
    _, _, s, rstd = mc2.mc2_add_rms_norm(x.cuda(), w.cuda(), r.cuda(), eps=EPS, need_rstd=True)
    s16 = s.cpu()  # the gradient is taken at the saved sum
    dx, dw = mc2.mc2_add_rms_norm_grad(dout.cuda(), s, w.cuda(), rstd, dsum.cuda())

    def loss(sv, wv):
        y = sv / torch.sqrt((sv * sv).mean(-1, keepdim=True) + EPS) * wv
        return (y * dout.double()).sum() + (sv * dsum.double()).sum()

    base, wd, d = s16.double(), w.double(), 1e-5
    for seed in range(4):
        v = rand(30 + seed, rows, h).double()
        num = (loss(base + d * v, wd) - loss(base - d * v, wd)) / (2 * d)
        # rounding of dx, and rstd having been taken before the sum was rounded (U relative)
        tol = (2 * U["bf16"] * (dx.cpu().double().abs() + 4.0) * v.abs()).sum() + 1e-6
        assert abs(num - (dx.cpu().double() * v).sum()) <= tol
        v = rand(40 + seed, h).double()
        num = (loss(base, wd + d * v) - loss(base, wd - d * v)) / (2 * d)
        tol = (2 * U["bf16"] * (dw.cpu().double().abs() + 4.0) * v.abs()).sum() + 1e-6
        assert abs(num - (dw.cpu().double() * v).sum()) <= tol


def test_norm_in_place_and_given_outputs(mc2):
    x, r, w = rand(50, 33, 1032), rand(51, 33, 1032), rand(52, 1032)
    want = mc2.mc2_add_rms_norm(x.cuda(), w.cuda(), r.cuda(), eps=EPS, need_rstd=True)
    xr, rr = x.cuda(), r.cuda()
    out = torch.empty_like(xr)
    got = mc2.mc2_add_rms_norm(xr, w.cuda(), rr, eps=EPS, need_rstd=True, out=out, sum_out=rr)
    assert got[0] is out and got[2] is rr
    for a, b in zip((want[0], want[2], want[3]), (got[0], got[2], got[3])):
        assert torch.equal(a, b)
    dout, dsum = rand(53, 33, 1032).cuda(), rand(54, 33, 1032).cuda()
    dx, dw = mc2.mc2_add_rms_norm_grad(dout, want[2], w.cuda(), want[3], dsum)
    dx2, dw2 = mc2.mc2_add_rms_norm_grad(dout, want[2], w.cuda(), want[3], dsum, dx=dsum)
    assert dx2 is dsum and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_norm_offsets_past_32_bits(mc2):
    """More than 2^31 elements: the last rows of a long batch."""
    rows, h = 262144 + 9, 8192
    x = torch.empty((rows, h), dtype=torch.bfloat16, device="cuda").fill_(0.5)
    tail = rand(60, 9, h)
    x[-9:] = tail.cuda()
    w = rand(61, h)
    out, _, _, rstd = mc2.mc2_add_rms_norm(x, w.cuda(), eps=EPS, need_rstd=True)
    _, ref_rstd, y = norm(tail, None, w, EPS)
    check(out[-9:], y, rounded(y, "bf16") + 1e-4 * y.abs(), "out")
    dx, _ = mc2.mc2_add_rms_norm_grad(out, x, w.cuda(), rstd)
    ref_dx, _ = norm_grad(out[-9:].cpu(), None, tail, w, rstd[-9:].cpu())
    check(dx[-9:], ref_dx, rounded(ref_dx, "bf16") + 1e-3, "dx")


def test_norm_same_bits_and_other_stream(mc2):
    x, r, w = rand(70, 700, 4096).cuda(), rand(71, 700, 4096).cuda(), rand(72, 4096).cuda()
    dout = rand(73, 700, 4096).cuda()
    a = mc2.mc2_add_rms_norm(x, w, r, need_rstd=True)
    ga = mc2.mc2_add_rms_norm_grad(dout, a[2], w, a[3])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = mc2.mc2_add_rms_norm(x, w, r, need_rstd=True, stream=st)
    gb = mc2.mc2_add_rms_norm_grad(dout, b[2], w, b[3], stream=st)
    st.synchronize()
    for u, v in zip((a[0], a[2], a[3], *ga), (b[0], b[2], b[3], *gb)):
        assert torch.equal(u, v)
