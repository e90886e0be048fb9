"""mc2_moe_route and its gradient against their definitions in 64 bits: the same experts, weights and gradients
within fp32's roundings (layer8_ref.score_error) and one rounding of the gradient's type."""
import math

import pytest
import torch

import layer8_ref as ref
from layer_ref import EPS32, TINY, U, check

pytestmark = pytest.mark.gpu
U32 = dict(U, f32=EPS32)
TINY32 = dict(TINY, f32=2.0 ** -126)


@pytest.fixture(scope="module")
def mc2():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd as m
    return m


def logits_of(seed, tokens, experts, dtype, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((tokens, experts), generator=g) * std).to(ref.LOGIT[dtype])


def run(mc2, l, top, bias=None, score="softmax", **kw):
    kinds = {"softmax": mc2.MC2_SCORE_SOFTMAX, "sigmoid": mc2.MC2_SCORE_SIGMOID}
    names = {"renorm": "renormalise"}
    ids, w = mc2.mc2_moe_route(l.cuda(), top, None if bias is None else bias.cuda(), score=kinds[score],
                               **{names.get(k, k): v for k, v in kw.items()})
    want, wr, _ = ref.route(l, top, bias, score, **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert torch.equal(ids.cpu(), want), (ids.cpu()[(ids.cpu() != want).any(1)][:3], want[(ids.cpu() != want).any(1)][:3])
    nan = torch.isnan(wr)
    assert torch.equal(torch.isnan(w.cpu()), nan)
    err = 2 * ref.score_error(l, score) + 16 * EPS32
    check(torch.where(nan, torch.zeros(()), w.cpu()), torch.where(nan, torch.zeros((), dtype=torch.float64), wr),
          torch.where(nan, 0.0, err * wr.abs() + 2.0 ** -126), "weights")
    return ids, w


@pytest.mark.parametrize("tokens,experts,top", [(1, 1, 1), (1, 5, 5), (3, 8, 2), (7, 63, 4), (4, 64, 64), (33, 65, 8),
                                                (5, 128, 6), (9, 160, 6), (130, 256, 8), (3, 257, 1), (6, 513, 63),
                                                (5, 1024, 8), (3, 1025, 16), (2, 2049, 8), (3, 4096, 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sizes(mc2, tokens, experts, top, dtype, score):
    print(f"route {tokens} x {experts} top {top} {dtype} {score}", flush=True)
    l = logits_of(tokens + experts, tokens, experts, dtype)
    run(mc2, l, top, None, score, renorm=True)
    run(mc2, l, top, None, score, renorm=False, scale=2.5)
    g = torch.Generator().manual_seed(experts)
    bias = torch.randn((experts,), generator=g) * 0.05
    run(mc2, l, top, bias, score, renorm=True, scale=-1.5)


@pytest.mark.parametrize("experts,groups,top_groups,top", [(8, 4, 2, 3), (64, 8, 3, 6), (160, 8, 3, 6), (256, 16, 6, 8),
                                                           (60, 5, 2, 7), (64, 64, 5, 5), (192, 64, 9, 20), (66, 33, 4, 3),
                                                           (1000, 8, 1, 8), (4096, 64, 7, 16), (4096, 2, 1, 8),
                                                           (4095, 63, 3, 64), (21, 7, 7, 21), (2050, 41, 4, 8)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(mc2, experts, groups, top_groups, top, group_top, score):
    if group_top > experts // groups:
        with pytest.raises(mc2.Mc2Error, match="group_top"):
            mc2.mc2_moe_route(torch.zeros((1, experts), device="cuda"), top, groups=groups, top_groups=top_groups,
                              group_top=group_top)
        return
    print(f"route groups {experts} / {groups} top {top_groups} {top} sum {group_top} {score}", flush=True)
    g = torch.Generator().manual_seed(groups)
    for dtype, biased in (("f32", False), ("f32", True), ("bf16", False), ("f16", True)):
        l = logits_of(experts + groups, 9, experts, dtype)
        bias = torch.randn((experts,), generator=g) * 0.1 if biased else None
        run(mc2, l, top, bias, score, groups=groups, top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lowest(mc2, score, bias):
    """Equal logits (and equal biases): experts in ascending order, groups too, in the fp32 and the fp64 choice."""
    for experts in (6, 64, 100, 300):
        b = torch.full((experts,), 0.25) if bias else None
        run(mc2, torch.zeros((3, experts)), 4, b, score)
        l = torch.zeros((4, experts))
        l[1, experts - 1] = 1.0
        l[2, ::2] = -1.0
        l[3, experts // 2:] = 0.5
        run(mc2, l, 5, b, score)
        run(mc2, -0.0 * torch.ones((2, experts)) + torch.tensor([[0.0], [-0.0]]), 3, b, score)
        run(mc2, l, 2, b, score, groups=2, top_groups=1, group_top=2)
        run(mc2, l, 2, b, score, groups=2, top_groups=1, group_top=1)
    zeros = torch.zeros((2, 8))
    zeros[0, 1::2] = -0.0
    zeros[1, ::2] = -0.0
    run(mc2, zeros, 3, None, score)


def test_near_ties_are_those_of_64_bits(mc2):
    """Scores + bias that differ by less than fp32 shows: the choice is still that of 64 bits."""
    g = torch.Generator().manual_seed(5)
    for score in ("softmax", "sigmoid"):
        for seed in range(6):
            l = logits_of(100 + seed, 40, 96, "f32", std=1.0)
            # a bias that cancels the first token's scores to within one part in 10^8 or so
            bias = (-ref.scores(l[:1].double(), score)[0]).float()
            l = l[:1].repeat(40, 1)
            l += torch.randn(l.shape, generator=g) * torch.logspace(-9, -3, 40)[:, None]
            run(mc2, l, 8, bias, score)
            run(mc2, l, 6, bias, score, groups=8, top_groups=3, group_top=2)


def test_a_bias_of_zeros(mc2):
    """Ties as 16-bit logits have them, under a bias that says nothing: the order of the logits, then of the experts."""
    for dtype in ("bf16", "f16", "f32"):
        l = logits_of(18, 300, 256, dtype, std=1.0)
        for score in ("softmax", "sigmoid"):
            ids, _ = run(mc2, l, 8, torch.zeros((256,)), score)
            plain, _ = run(mc2, l, 8, None, score)
            assert torch.equal(ids, plain)
            run(mc2, l, 8, torch.zeros((256,)), score, groups=16, top_groups=5, group_top=2)
            run(mc2, l, 20, torch.zeros((256,)), score)


def test_bias_that_swamps_the_scores(mc2):
    l = logits_of(6, 20, 70, "f32")
    run(mc2, l, 5, torch.full((70,), 1e7), "sigmoid")
    b = torch.full((70,), 4096.0)
    b[::3] = 4097.0
    run(mc2, l, 5, b, "softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_that_are_off(mc2, score):
    """-inf logits, -inf and NaN biases, +inf ones; tokens with too few experts, and with none."""
    l = logits_of(7, 12, 40, "f32")
    l[:, 3] = -math.inf
    l[1] = -math.inf
    l[2] = -math.inf
    l[2, 17] = -60.0
    l[3, 2:] = -math.inf
    run(mc2, l, 4, None, score)
    run(mc2, l, 4, None, score, renorm=False)
    b = torch.zeros((40,))
    b[0], b[5], b[9] = -math.inf, math.nan, math.inf
    run(mc2, l, 4, b, score)
    for group_top in (1, 2):
        run(mc2, l, 4, None, score, groups=8, top_groups=2, group_top=group_top)
        run(mc2, l, 4, b, score, groups=8, top_groups=2, group_top=group_top)
    ids, w = run(mc2, torch.full((2, 8), -math.inf), 2, None, score)
    assert (ids == -1).all() and torch.count_nonzero(w) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_at_the_ends_of_the_type(mc2, score):
    """A group's two scores of the lowest or the largest bias have a sum past fp32: lower or higher than any one of them,
    and a group still."""
    low, big = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    for experts, groups, top in ((32, 4, 16), (32, 4, 9), (96, 8, 30), (512, 8, 64)):
        per = experts // groups
        l = logits_of(experts + top, 6, experts, "f32")
        for value in (low, big, -math.inf):
            bias = torch.full((experts,), value)
            bias[per:2 * per] = 0.0                      # one group at its scores
            run(mc2, l, top, bias, score, groups=groups, top_groups=max(2, -(-top // per)), group_top=2)
            bias[3 * per:4 * per - 1] = -math.inf        # one with a single expert: its value is not a sum
            run(mc2, l, top, bias, score, groups=groups, top_groups=max(2, -(-top // per)), group_top=2)
            bias[2 * per] = 0.75 * value                 # sums that differ past fp32's range
            run(mc2, l, top, bias, score, groups=groups, top_groups=max(2, -(-top // per)), group_top=2)


def test_nan_and_infinity(mc2):
    l = logits_of(8, 6, 33, "f32")
    l[1, 32] = math.nan
    l[2, 0] = math.inf
    l[3, 5], l[3, 6] = math.nan, -math.inf
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.linspace(0, 0.1, 33)):
            ids, w = run(mc2, l, 3, bias, score)
            assert (ids[1] == -1).all() and torch.isnan(w[1]).all() and (ids[0] >= 0).all()
    # far logits: scores of 0, and sums of them
    far = torch.tensor([[-300.0, -310.0, -400.0, -1e30], [300.0, 200.0, -200.0, 1e30], [1e38, -1e38, 3e38, -3e38]])
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, w = mc2.mc2_moe_route(far.cuda(), 2, score=["softmax", "sigmoid"].index(score), renormalise=renorm)
            assert torch.equal(ids.cpu(), ref.route(far, 2, None, score)[0])
            assert torch.isfinite(w).all() and (w >= 0).all() and (w <= 1).all()


def test_shares_of_experts_far_below_the_others(mc2):
    """The kept group's logits are so far below the best one that its scores are 0 in fp32: their shares are not."""
    l = torch.tensor([[0.0, -1.0, -500.0, -501.0], [3.0, 3.0, -1e4, -1e4]])
    bias = torch.tensor([0.0, 0.0, 5.0, 5.0])
    ids, w = run(mc2, l, 2, bias, "softmax", groups=2, top_groups=1, group_top=2)
    assert torch.equal(ids.cpu(), torch.tensor([[2, 3], [2, 3]], dtype=torch.int32))
    share = torch.sigmoid(torch.tensor([1.0, -1.0], dtype=torch.float64))
    check(w[0].cpu(), share, 32 * EPS32 * share, "shares")
    assert torch.equal(w[1].cpu(), torch.tensor([0.5, 0.5]))
    got = mc2.mc2_moe_route_grad(torch.tensor([[1.0, 0.0], [1.0, 0.0]]).cuda(), l.cuda(), ids)
    want = torch.tensor([float(share[0] * share[1]), 0.25], dtype=torch.float64)
    check(got[:, 2].cpu(), want, 64 * EPS32 * want, "gradient")


def test_no_tokens_outputs_given_and_streams(mc2):
    ids, w = mc2.mc2_moe_route(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert mc2.mc2_moe_route_grad(w, torch.empty((0, 8), device="cuda"), ids).shape == (0, 8)
    l = logits_of(9, 50, 64, "bf16").cuda()
    a, b = mc2.mc2_moe_route(l, 4)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ids, w = torch.empty_like(a), torch.empty_like(b)
    got = mc2.mc2_moe_route(l, 4, expert_ids=ids, weights=w, stream=st)
    st.synchronize()
    assert got[0] is ids and got[1] is w and torch.equal(ids, a) and torch.equal(w, b)
    d = torch.randn((50, 4), device="cuda")
    want = mc2.mc2_moe_route_grad(d, l, a)
    st.wait_stream(torch.cuda.current_stream())
    got = mc2.mc2_moe_route_grad(d, l, a, stream=st)
    st.synchronize()
    assert torch.equal(want, got)
    again = mc2.mc2_moe_route_grad(d, l, a, dlogits=l)  # in place
    assert again is l and torch.equal(want, l)


# ------------------------------------------------------------------ gradient
def run_grad(mc2, l, ids, dw, score, renorm, scale=1.0):
    got = mc2.mc2_moe_route_grad(dw.cuda(), l.cuda(), ids.cuda(), score=["softmax", "sigmoid"].index(score),
                                 renormalise=renorm, scale=scale)
    want, size = ref.route_grad(dw, l, ids, score, renorm, scale)
    assert got.dtype == l.dtype
    dt = {v: k for k, v in ref.LOGIT.items()}[l.dtype]
    # terms with up to four factors of a score's error each, and sums over the choices
    err = (4 * ref.score_error(l, score) + (ids.shape[1] + 16) * EPS32) * size
    check(got, want, U32[dt] * want.abs() + (1 + U32[dt]) * err + TINY32[dt], "dlogits")
    return got


@pytest.mark.parametrize("tokens,experts,top", [(1, 1, 1), (2, 5, 3), (3, 64, 4), (33, 65, 8), (9, 160, 6), (70, 256, 8),
                                                (4, 513, 64), (3, 1025, 16), (2, 4096, 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_grad_sizes(mc2, tokens, experts, top, dtype):
    print(f"route_grad {tokens} x {experts} top {top} {dtype}", flush=True)
    l = logits_of(11 + experts, tokens, experts, dtype)
    dw = torch.randn((tokens, top), generator=torch.Generator().manual_seed(top))
    for score in ("softmax", "sigmoid"):
        ids = ref.route(l, top, None, score)[0]
        for renorm in (False, True):
            run_grad(mc2, l, ids, dw, score, renorm, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_grad_of_missing_choices(mc2, score, renorm):
    """Ids of -1 or past the experts, whatever their dweights hold; the same expert twice; off experts."""
    l = logits_of(12, 8, 20, "f32")
    l[:, 7] = -math.inf
    l[4] = -math.inf
    ids = ref.route(l, 4, None, score)[0]
    dw = torch.randn((8, 4), generator=torch.Generator().manual_seed(1))
    ids[0, 2], ids[1], ids[2, 0], ids[3, 1] = -1, -1, 20, 2 ** 31 - 1
    dw[0, 2] = math.nan
    dw[1, 0], dw[2, 0] = math.inf, math.nan
    ids[5, 3] = ids[5, 0]
    got = run_grad(mc2, l, ids, dw, score, renorm)
    assert torch.count_nonzero(got[1]) == 0 and torch.count_nonzero(got[4]) == 0 and torch.isfinite(got).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_grad_against_differences(mc2, score, renorm):
    """The weights of a fixed choice move with the logits as the gradient says."""
    l = logits_of(13, 6, 24, "f32")
    dw = torch.randn((6, 3), generator=torch.Generator().manual_seed(2))
    kind = ["softmax", "sigmoid"].index(score)
    ids, _ = mc2.mc2_moe_route(l.cuda(), 3, score=kind, renormalise=renorm, scale=2.0)
    got = mc2.mc2_moe_route_grad(dw.cuda(), l.cuda(), ids, score=kind, renormalise=renorm, scale=2.0).cpu().double()

    def loss(v):
        w = ref.scores(v, score).gather(1, ids.cpu().long())
        return (2.0 * (w / w.sum(1, keepdim=True) if renorm else w) * dw.double()).sum()

    step = 1e-5
    for i in range(8):
        v = torch.randn(l.shape, generator=torch.Generator().manual_seed(20 + i)).double()
        num = (loss(l.double() + step * v) - loss(l.double() - step * v)) / (2 * step)
        # fp32's roundings of the gradient; the differences' own error is step^2 times a third derivative below 8
        assert abs(num - (got * v).sum()) <= (64 * EPS32 * (1 + got.abs()) * v.abs()).sum() + 1e-8, (score, renorm, i)


def test_graph_replay(mc2):
    """Router and gradient in one captured graph, replayed on new logits with eager work between."""
    l = logits_of(14, 300, 96, "f32").cuda()
    bias = (torch.linspace(-0.1, 0.1, 96)).cuda()
    dw = torch.randn((300, 6), device="cuda")
    kw = dict(score=mc2.MC2_SCORE_SIGMOID, groups=8, top_groups=3, group_top=2)

    def both():
        ids, w = mc2.mc2_moe_route(l, 6, bias, **kw)
        return ids, w, mc2.mc2_moe_route_grad(dw, l, ids, score=mc2.MC2_SCORE_SIGMOID)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in (15, 16, 17):
        l.copy_(logits_of(seed, 300, 96, "f32"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, both()):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ the ends of the scores
FAR = [[-88.0, -89.0, -200.0, -300.0], [-95.0, -96.0, -97.0, -500.0], [-103.0, -104.0, -110.0, -105.5],
       [-300.0, -310.0, -400.0, -1e30], [-740.0, -700.5, -710.0, -720.0], [0.5, -88.5, -120.0, -130.0],
       [-20.0, -90.0, -95.0, -1e4], [-800.0, -801.0, -1e30, -math.inf], [-1e30, -2e30, -3e38, -math.inf]]


@pytest.mark.parametrize("scale", [1.0, -1.5])
def test_sigmoids_far_below_one(mc2, scale):
    """Logits whose sigmoids are subnormal or 0 in fp32: their shares are those of 64 bits, and so are the shares'
    gradients; the scores themselves are right down to fp32's last subnormal numbers.

    A share is a quotient of exp(d) / (1 + exp(l)), d a difference to the largest of the chosen (or 0), rounded: |d|
    half steps; an exponential is within 4, the other factor 6, the product 1, the sum 2, for a share twice that and 2
    for quotient and scale: 32 + 2 |d|.  A score alone has no sum: 16, and three roundings of half a subnormal step."""
    l = torch.tensor(FAR)
    d = torch.tensor([1.0, 1.0, 1.0, 10.0, 9.5, 88.5, 70.0, 0.0, 0.0], dtype=torch.float64)[:, None]
    for renorm in (True, False):
        ids, w = mc2.mc2_moe_route(l.cuda(), 2, score=mc2.MC2_SCORE_SIGMOID, renormalise=renorm, scale=scale)
        want, wr, _ = ref.route(l, 2, None, "sigmoid", renorm=renorm, scale=scale)
        assert torch.equal(ids.cpu(), want)
        err = (32 + 2 * d) * EPS32 * wr.abs() if renorm else 16 * EPS32 * wr.abs()
        check(w, wr, err + 2.0 ** -148, f"weights, renormalise={renorm}")
        dw = torch.tensor([[1.0, -0.5]]).repeat(len(FAR), 1)
        got = mc2.mc2_moe_route_grad(dw.cuda(), l.cuda(), ids, score=mc2.MC2_SCORE_SIGMOID, renormalise=renorm,
                                     scale=scale)
        grad, size = ref.route_grad(dw, l, want, "sigmoid", renorm, scale)
        check(got, grad, (96 + 4 * d) * EPS32 * size + 2.0 ** -126, f"gradient, renormalise={renorm}")


def test_groups_whose_scores_cancel(mc2):
    """A group's two values of opposite signs: their sum is small, and its error that of the large values."""
    p = torch.tensor([0.54, 0.50, 0.53, 0.52])
    big = torch.tensor([1e6, -1e6, 1e6, -1e6])
    ids, _ = run(mc2, torch.log(p / (1 - p))[None], 2, big, "sigmoid", groups=2, top_groups=1, group_top=2)
    assert ids.tolist() == [[2, 3]]
    for score in ("sigmoid", "softmax"):
        for seed, size in enumerate((128.0, 1000.0, 3e4, 1e6)):
            # 16 and 64 lanes a token; 2 experts a group, or 4 of which two hold the large values
            for experts, groups in ((128, 64), (256, 64), (384, 64)):
                l = logits_of(seed + experts, 120, experts, "f32")
                bias = torch.zeros((groups, experts // groups))
                bias[:, 0], bias[:, 1:] = size, -size
                run(mc2, l, 6, bias.flatten(), score, groups=groups, top_groups=5, group_top=2)


def test_saturated_sigmoids_without_a_bias(mc2):
    """Logits whose sigmoids are equal even in 64 bits: without a bias the order is the logits' own, with one (of zeros)
    the scores tie and the lowest expert comes first."""
    l = torch.tensor([[40.0, 41.0, 39.0, 45.0], [-1000.0, -999.0, -2000.0, -998.0]])
    ids, _ = run(mc2, l, 2, None, "sigmoid")
    assert ids.tolist() == [[3, 1], [3, 1]]
    ids, _ = run(mc2, l, 2, torch.zeros((4,)), "sigmoid")
    assert ids.tolist() == [[0, 1], [0, 1]]
    # groups by their best logit go the same way, also for a token whose many equal logits are settled in 64 bits
    for score in ("sigmoid", "softmax"):
        l = torch.linspace(1.0, 2.0, 32).repeat(2, 1)
        l[:, 0], l[:, 16] = 40.0, 41.0
        l[1, 17:] = 1.0
        if score == "softmax":
            l[:, 1:16] -= 900.0
            l[:, 0], l[:, 16:] = -800.0, l[:, 16:] - 840.0  # both groups' scores are 0 in 64 bits beside the third's
            l = torch.cat([l, torch.zeros((2, 16))], dim=1)
        kind = [mc2.MC2_SCORE_SOFTMAX, mc2.MC2_SCORE_SIGMOID][score == "sigmoid"]
        ids, _ = mc2.mc2_moe_route(l.cuda(), 19 if score == "softmax" else 3, score=kind, groups=l.shape[1] // 16,
                                   top_groups=l.shape[1] // 16 - 1, group_top=1)
        first = list(range(32, 48)) if score == "softmax" else []
        assert ids[0].tolist() == first + [16, 31, 30] and ids[1].tolist() == first + [16, 17, 18], score


def test_tokens_whose_nan_is_kept(mc2):
    """keep_nan: a token without a usable logit has the first experts and NaN weights; nothing else changes."""
    for experts, top in ((33, 3), (300, 20)):
        l = logits_of(experts, 9, experts, "f32")
        l[1, 32], l[2, 0], l[4, 5], l[6] = math.nan, math.inf, -math.inf, -math.inf
        for score in (mc2.MC2_SCORE_SOFTMAX, mc2.MC2_SCORE_SIGMOID):
            ids, w = mc2.mc2_moe_route(l.cuda(), top, score=score)
            kept, wk = mc2.mc2_moe_route(l.cuda(), top, score=score, keep_nan=True)
            nan = torch.isnan(w).all(1)
            assert nan.tolist() == [r == 1 or (r == 2 and score == 0) for r in range(9)]
            assert (ids[nan] == -1).all() and torch.equal(kept[~nan], ids[~nan]) and (ids[6] == -1).all()
            assert torch.equal(w[~nan], wk[~nan]) and torch.isnan(wk[nan]).all()
            assert (kept[nan] == torch.arange(top, device="cuda", dtype=torch.int32)).all()
