"""mc2_moe_permute, mc2_moe_unpermute and the gradients against plain loops and 64-bit sums.

Row order, maps and ranges are exact; a weighted sum of `top` products in fp32
is within (top + 1) roundings of its terms' sizes, plus the output's own.
"""
import pytest
import torch

from layer_ref import DT, EPS32, check, rand, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


def make_ids(seed, tokens, top, experts, drop=0.1, skew=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, experts, (tokens, top), generator=g, dtype=torch.int32)
    if skew:
        ids = torch.where(torch.rand((tokens, top), generator=g) < 0.7, torch.zeros_like(ids), ids)
    bad = torch.where(torch.rand((tokens, top), generator=g) < 0.5, torch.tensor(-1), torch.tensor(experts)).int()
    return torch.where(torch.rand((tokens, top), generator=g) < drop, bad, ids)


def plain_map(ids, experts):
    """(row_map, offsets, kept choices in order) by a stable sort in Python."""
    flat = ids.reshape(-1).tolist()
    order = sorted((e, i) for i, e in enumerate(flat) if 0 <= e < experts)
    row_map = torch.full((len(flat),), -1, dtype=torch.int32)
    for r, (_, i) in enumerate(order):
        row_map[i] = r
    counts = [0] * experts
    for e, _ in order:
        counts[e] += 1
    offsets = torch.tensor([0] + counts).cumsum(0).int()
    return row_map.view(ids.shape), offsets, [i for _, i in order]


SORTS = [(1, 1, 1), (1, 4, 8), (3, 2, 5), (64, 1, 64), (65, 3, 7), (1000, 2, 160), (4096, 2, 8), (4097, 2, 64),
         (8191, 4, 32), (20000, 1, 512), (5000, 8, 513), (3000, 3, 4096), (1, 1, 4096)]


@pytest.mark.parametrize("tokens,top,experts", SORTS)
@pytest.mark.parametrize("skew", [False, True])
def test_permute(mc2, tokens, top, experts, skew):
    print(f"permute tokens={tokens} top={top} experts={experts} skew={skew}", flush=True)
    h = 24
    x = rand(1, tokens, h)
    ids = make_ids(2 + tokens, tokens, top, experts, skew=skew)
    out, row_map, offsets = mc2.mc2_moe_permute(x.cuda(), ids.cuda(), experts)
    want_map, want_offsets, order = plain_map(ids, experts)
    assert torch.equal(row_map.cpu(), want_map)
    assert torch.equal(offsets.cpu(), want_offsets)
    want = torch.zeros((tokens * top, h), dtype=x.dtype)
    want[:len(order)] = x[torch.tensor(order, dtype=torch.long) // top]
    assert torch.equal(out.cpu(), want)


# choices on both sides of 256 and of 1024, many per token, more experts than choices
FEW = [(64, 4, 160), (257, 1, 4096), (128, 8, 32), (205, 5, 64), (2, 500, 3), (1, 64, 64), (1024, 1, 963)]


@pytest.mark.parametrize("tokens,top,experts", FEW)
@pytest.mark.parametrize("h", [7, 264, 2056])
def test_permute_few(mc2, tokens, top, experts, h):
    print(f"permute tokens={tokens} top={top} experts={experts} h={h}", flush=True)
    x, ids = rand(30, tokens, h), make_ids(31 + tokens, tokens, top, experts, drop=0.2)
    out, row_map, offsets = mc2.mc2_moe_permute(x.cuda(), ids.cuda(), experts)
    want_map, want_offsets, order = plain_map(ids, experts)
    assert torch.equal(row_map.cpu(), want_map)
    assert torch.equal(offsets.cpu(), want_offsets)
    want = torch.zeros((tokens * top, h), dtype=x.dtype)
    want[:len(order)] = x[torch.tensor(order, dtype=torch.long) // top]
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("h", [1, 5, 8, 63, 64, 1000, 2048, 2056, 4096, 7168])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_permute_widths(mc2, h, dtype):
    x, ids = rand(3, 37, h, dtype=dtype), make_ids(4, 37, 3, 6, drop=0.3)
    out, row_map, _ = mc2.mc2_moe_permute(x.cuda(), ids.cuda(), 6)
    _, _, order = plain_map(ids, 6)
    want = torch.zeros((111, h), dtype=x.dtype)
    want[:len(order)] = x[torch.tensor(order, dtype=torch.long) // 3]
    assert torch.equal(out.cpu(), want)


def test_permute_nothing_kept_and_no_tokens(mc2):
    x = rand(5, 40, 16)
    out, row_map, offsets = mc2.mc2_moe_permute(x.cuda(), torch.full((40, 2), -1, dtype=torch.int32).cuda(), 9)
    assert torch.count_nonzero(out.cpu()) == 0 and torch.all(row_map.cpu() == -1) and torch.all(offsets.cpu() == 0)
    out = mc2.mc2_moe_unpermute(out, row_map, torch.ones((40, 2), device="cuda"))
    assert torch.count_nonzero(out.cpu()) == 0
    empty = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    out, row_map, offsets = mc2.mc2_moe_permute(empty, torch.empty((0, 2), dtype=torch.int32, device="cuda"), 9)
    assert out.shape == (0, 16) and row_map.shape == (0, 2) and torch.all(offsets.cpu() == 0)
    assert mc2.mc2_moe_unpermute(empty, row_map).shape == (0, 16)
    dy, dw = mc2.mc2_moe_unpermute_grad(empty, torch.ones((5, 16), dtype=torch.bfloat16, device="cuda"), row_map)
    assert torch.count_nonzero(dy.cpu()) == 0 and dw.shape == (0, 2)


def plain_unpermute(y, row_map, weights):
    tokens, top = row_map.shape
    out, size = torch.zeros((tokens, y.shape[1]), dtype=torch.float64), torch.zeros((tokens, y.shape[1]), dtype=torch.float64)
    for t in range(tokens):
        for j in range(top):
            r = int(row_map[t, j])
            if 0 <= r < y.shape[0]:
                term = y[r].double() * (1.0 if weights is None else float(weights[t, j]))
                out[t] += term
                size[t] += term.abs()
    return out, size


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,top,h", [(1, 1, 1), (1, 8, 4096), (5, 2, 7), (16, 4, 4096), (33, 3, 1000), (9, 5, 63),
                                          (130, 6, 200), (21, 9, 2056)])
@pytest.mark.parametrize("weighted", [True, False])
def test_unpermute_and_gradient(mc2, tokens, top, h, dtype, weighted):
    print(f"unpermute tokens={tokens} top={top} h={h} {dtype} weights={weighted}", flush=True)
    ids = make_ids(7 + tokens, tokens, top, 11, drop=0.25)
    row_map, _, order = plain_map(ids, 11)
    y, dout = rand(8, tokens * top, h, dtype=dtype), rand(9, tokens, h, dtype=dtype)
    weights = torch.rand((tokens, top), generator=torch.Generator().manual_seed(10)) if weighted else None
    wc = None if weights is None else weights.cuda()
    out = mc2.mc2_moe_unpermute(y.cuda(), row_map.cuda(), wc)
    ref, size = plain_unpermute(y, row_map, weights)
    check(out, ref, rounded(ref, dtype) + (top + 1) * EPS32 * size, "out")

    dy, dw = mc2.mc2_moe_unpermute_grad(dout.cuda(), y.cuda(), row_map.cuda(), wc)
    ref_dy = torch.zeros(y.shape, dtype=torch.float64)
    ref_dw, dw_size = torch.zeros((tokens, top), dtype=torch.float64), torch.zeros((tokens, top), dtype=torch.float64)
    for t in range(tokens):
        for j in range(top):
            r = int(row_map[t, j])
            if r >= 0:
                ref_dy[r] = dout[t].double() * (1.0 if weights is None else float(weights[t, j]))
                p = y[r].double() * dout[t].double()
                ref_dw[t, j], dw_size[t, j] = p.sum(), p.abs().sum()
    check(dy, ref_dy, rounded(ref_dy, dtype) + EPS32 * ref_dy.abs(), "dy")
    check(dw, ref_dw, (h / 64 + 32) * EPS32 * dw_size, "dweights")
    only, none = mc2.mc2_moe_unpermute_grad(dout.cuda(), y.cuda(), row_map.cuda(), wc, need_dweights=False)
    assert none is None and torch.equal(only, dy)


def test_unpermute_ignores_rows_outside(mc2):
    y = rand(11, 6, 40)
    row_map = torch.tensor([[0, 6], [-7, 5], [2 ** 31 - 1, 3]], dtype=torch.int32)
    out = mc2.mc2_moe_unpermute(y.cuda(), row_map.cuda())
    assert torch.equal(out.cpu(), y[[0, 5, 3]])


def test_unpermute_is_the_gradient_of_permute(mc2):
    """<permute(x), d> == <x, unpermute(d)> with integer values, exactly."""
    g = torch.Generator().manual_seed(12)
    x = torch.randint(-4, 5, (50, 32), generator=g).bfloat16()
    d = torch.randint(-4, 5, (150, 32), generator=g).bfloat16()
    ids = make_ids(13, 50, 3, 4, drop=0.2)
    out, row_map, _ = mc2.mc2_moe_permute(x.cuda(), ids.cuda(), 4)
    dx = mc2.mc2_moe_unpermute(d.cuda(), row_map)
    assert (out.cpu().double() * d.double()).sum() == (x.double() * dx.cpu().double()).sum()


def test_unpermute_grad_differences(mc2):
    """dy and dweights against differences of the weighted sum (linear in each, so exact up to rounding)."""
    ids = make_ids(14, 12, 2, 3, drop=0.2)
    row_map, _, _ = plain_map(ids, 3)
    y, dout = rand(15, 24, 16), rand(16, 12, 16)
    weights = torch.rand((12, 2), generator=torch.Generator().manual_seed(17)).double()
    dy, dw = mc2.mc2_moe_unpermute_grad(dout.cuda(), y.cuda(), row_map.cuda(), weights.float().cuda())

    def loss(yv, wv):
        out = torch.zeros((12, 16), dtype=torch.float64)
        for t in range(12):
            for j in range(2):
                if row_map[t, j] >= 0:
                    out[t] += wv[t, j] * yv[int(row_map[t, j])]
        return (out * dout.double()).sum()

    v = rand(18, 24, 16).double()
    num = (loss(y.double() + v, weights) - loss(y.double() - v, weights)) / 2
    assert abs(num - (dy.cpu().double() * v).sum()) <= (2.0 ** -8 * dy.cpu().double().abs() * v.abs()).sum() + 1e-6
    v = rand(19, 12, 2).double()
    num = (loss(y.double(), weights + v) - loss(y.double(), weights - v)) / 2
    assert abs(num - (dw.cpu().double() * v).sum()) <= 1e-4


def test_rows_past_32_bits(mc2):
    """Row offsets beyond 2^31 elements, read and written."""
    rows, h = 262144 + 8, 8192
    y = torch.zeros((rows, h), dtype=torch.bfloat16, device="cuda")
    tail = rand(20, 8, h)
    y[-8:] = tail.cuda()
    row_map = torch.arange(rows - 8, rows, dtype=torch.int32).view(4, 2)
    out = mc2.mc2_moe_unpermute(y, row_map.cuda())
    ref, size = plain_unpermute(tail, row_map - (rows - 8), None)
    check(out, ref, rounded(ref, "bf16") + 3 * EPS32 * size, "out")
    del y
    # permute writes them: all tokens to one expert but the last ones, which follow
    x = torch.zeros((rows // 2, h), dtype=torch.bfloat16, device="cuda")
    x[-1] = tail[0].cuda()
    ids = torch.zeros((rows // 2, 2), dtype=torch.int32, device="cuda")
    ids[-1] = 1
    out, row_map, offsets = mc2.mc2_moe_permute(x, ids, 2)
    assert offsets.tolist() == [0, rows - 2, rows] and row_map[-1].tolist() == [rows - 2, rows - 1]
    assert torch.equal(out[-2:].cpu(), tail[:1].expand(2, h))
    del x
    dy, _ = mc2.mc2_moe_unpermute_grad(torch.cat([torch.zeros((rows // 2 - 1, h), dtype=torch.bfloat16, device="cuda"),
                                                  tail[:1].cuda()]), out, row_map)
    assert torch.equal(dy[-2:].cpu(), tail[:1].expand(2, h))


def test_same_bits_and_other_stream(mc2):
    x, ids = rand(21, 9000, 512).cuda(), make_ids(22, 9000, 4, 64).cuda()
    weights = torch.rand((9000, 4), generator=torch.Generator().manual_seed(23)).cuda()
    a = mc2.mc2_moe_permute(x, ids, 64)
    ga = mc2.mc2_moe_unpermute_grad(x, a[0], a[1], weights)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = mc2.mc2_moe_permute(x, ids, 64, stream=st)
    gb = mc2.mc2_moe_unpermute_grad(x, b[0], b[1], weights, stream=st)
    u = mc2.mc2_moe_unpermute(b[0], b[1], weights, stream=st)
    st.synchronize()
    for p, q in zip((*a, *ga, mc2.mc2_moe_unpermute(a[0], a[1], weights)), (*b, *gb, u)):
        assert torch.equal(p, q)
