"""The router and the 8-bit operators on tensors of more than 2^31 elements, and on more rows than one launch takes:
their first rows, those about the 2^31st element and their last ones against the same rows alone, which the other
tests hold against 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def places(rows, cols):
    """Pieces of 40 rows: the first, those with element 2^31 (of the codes and of the 16-bit bytes), the last."""
    at = [0, (1 << 30) // cols - 20, (1 << 31) // cols - 20, (1 << 21) - 20, rows - 40]
    return [slice(a, a + 40) for a in at if 0 <= a <= rows - 40]


def some(rows, cols, dtype, seed=1):
    """(rows, cols) of zeros with random values in the pieces."""
    x = torch.zeros((rows, cols), dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    for p in places(rows, cols):
        if dtype == torch.int8:
            x[p] = torch.randint(-127, 128, (40, cols), generator=g, device="cuda", dtype=dtype)
        else:
            x[p] = torch.randn((40, cols), generator=g, device="cuda").to(dtype)
    return x


@pytest.mark.parametrize("rows,cols,group", [((1 << 21) + 70, 1040, 0), ((1 << 21) + 70, 1039, 128),
                                             ((1 << 23) + 70, 4100, 0)])
def test_codes(mc2, rows, cols, group):
    print(f"codes {rows} x {cols} group {group}", flush=True)
    x = some(rows, cols, torch.bfloat16)
    codes, scale = mc2.mc2_quant_rows(x, group=group)
    want = [mc2.mc2_quant_rows(x[p].clone(), group=group) for p in places(rows, cols)]
    del x
    out = mc2.mc2_dequant_rows(codes, scale, group=group)
    for p, (c, s) in zip(places(rows, cols), want):
        assert torch.equal(codes[p], c) and torch.equal(scale[p], s)
        assert torch.equal(out[p], mc2.mc2_dequant_rows(c, s, group=group)) and c.any()


def test_router(mc2):
    tokens, experts = (1 << 20) + 70, 2080
    l = some(tokens, experts, torch.bfloat16)
    ids, w = mc2.mc2_moe_route(l, 8, score=mc2.MC2_SCORE_SIGMOID)
    dl = mc2.mc2_moe_route_grad(w, l, ids, score=mc2.MC2_SCORE_SIGMOID)
    for p in places(tokens, experts):
        one = l[p].clone()
        i, v = mc2.mc2_moe_route(one, 8, score=mc2.MC2_SCORE_SIGMOID)
        assert torch.equal(ids[p], i) and torch.equal(w[p], v)
        assert torch.equal(dl[p], mc2.mc2_moe_route_grad(v, one, i, score=mc2.MC2_SCORE_SIGMOID))


@pytest.mark.parametrize("k", [4096, 4100, 4097])
def test_linear(mc2, k):
    """x past 2^31 codes; then w, in groups."""
    m, n = (1 << 19) + 4000, 72
    g = torch.Generator(device="cuda").manual_seed(k)
    x, xs = some(m, k, torch.int8), torch.rand((m,), generator=g, device="cuda")
    w = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand((n,), generator=g, device="cuda") * 1e-3
    out = mc2.mc2_linear_i8(x, xs, w, ws)
    for p in places(m, k):
        assert torch.equal(out[p], mc2.mc2_linear_i8(x[p].clone(), xs[p].clone(), w, ws))
    del x, out
    groups, n = 65, 8192
    w = torch.zeros((groups, n, k), dtype=torch.int8, device="cuda")
    for e in (0, groups - 1):
        w[e] = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand((groups, n), generator=g, device="cuda") * 1e-3
    x = torch.randint(-127, 128, (130, k), generator=g, device="cuda", dtype=torch.int8)
    offsets = torch.arange(0, 2 * groups + 1, 2, dtype=torch.int32, device="cuda")
    out = mc2.mc2_linear_i8(x, xs[:130], w, ws, group_offsets=offsets)
    assert not out[2:128].any()
    for e in (0, groups - 1):
        p = slice(2 * e, 2 * e + 2)
        assert torch.equal(out[p], mc2.mc2_linear_i8(x[p].clone(), xs[p].clone(), w[e], ws[e])) and out[p].any()


def test_gradient(mc2):
    """z and dout past 2^31 elements: dx of pieces; dw and dbias of a dout that has nothing outside them."""
    m, k, n = (1 << 18) + 70, 64, 8256
    z, dout = some(m, n, torch.int8, 2), some(m, n, torch.bfloat16, 3)
    x = some(m, k, torch.int8, 4)
    pieces = places(m, n)
    g = torch.Generator(device="cuda").manual_seed(5)
    zs = torch.rand((m, -(-n // 128)), generator=g, device="cuda") * 0.02
    xs = torch.rand((m, 1), generator=g, device="cuda") * 0.02
    for p in pieces:
        x[p] = torch.randint(-127, 128, (40, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randn((n, k), generator=g, device="cuda").to(torch.bfloat16)
    kw = dict(act=mc2.MC2_ACT_RELU, need_dbias=True)
    dx, dw, db = mc2.mc2_linear_act_grad_i8(dout, x, xs, w, z, zs, **kw)
    cat = lambda t: torch.cat([t[p] for p in pieces])
    dx1, dw1, db1 = mc2.mc2_linear_act_grad_i8(cat(dout), cat(x), cat(xs), w, cat(z), cat(zs), **kw)
    # Sums of the same terms in another order (of n in parts, for the few rows alone; among zeros): an addition's half
    # step for each on either side, of all their magnitudes at most, and one rounding of either result.
    def near(got, want, terms, size):
        want = want.float()
        assert ((got.float() - want).abs() <= 2.01 * 2.0 ** -8 * want.abs() + 2 * terms * 2.0 ** -24 * size).all()
        assert want.any()

    rows, top = 40 * len(pieces), cat(dout).float().abs().max()
    near(cat(dx), dx1, n, cat(dout).float().abs() @ w.float().abs())
    near(dw, dw1, rows, rows * 127 * 0.02 * top)
    near(db, db1, rows, rows * top)
