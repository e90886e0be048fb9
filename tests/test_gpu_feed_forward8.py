"""The feed-forward modules with their activations kept in 8 bits, with mc2_moe_route's choice, and served in int8,
end to end: against 64 bits, against the 16-bit modules, and call by call."""
import pytest
import torch

import layer8_ref as ref
from layer_ref import U, act
from test_gpu_feed_forward import leaf, near, norm64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ff():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd.feed_forward as m
    return m


def at_codes(value, kept):
    """A tensor whose value is `kept` and whose gradient goes to `value` (rounding to codes has the slope 1)."""
    return value + (kept - value).detach()


def kept_values(mc2, t):
    c, s = mc2.mc2_quant_rows(t, group=128)
    return ref.values(c.cpu(), s.cpu(), 128)


def test_kept_feed_forward_trains(ff):
    """The forward is the 16-bit one bit for bit; the gradients are those of the formula with the first linear's input
    and pre-activation at their codes' values (near()'s bound)."""
    import comm_matmul_tensor_amd as mc2
    torch.manual_seed(1)
    plain, block = ff.FeedForward(192, 520), ff.FeedForward(192, 520, keep8=True)
    block.load_state_dict(plain.state_dict())
    with torch.no_grad():
        for b in (plain, block):
            b.b1.copy_(torch.linspace(-0.5, 0.5, 520))
    x = torch.randn((77, 192), device="cuda").bfloat16().requires_grad_()
    d = torch.randn((77, 192), device="cuda").bfloat16()
    out = block(x)
    assert torch.equal(out, plain(x)) and torch.equal(out, block.eval()(x))
    with torch.no_grad():
        assert torch.equal(out, block(x))
        y = mc2.mc2_add_rms_norm(x, block.norm)[0]
        z = mc2.mc2_linear_act(y, block.w1, block.b1, act=block.act, need_z=True)[1]
    out.backward(d)
    p = {k: leaf(v) for k, v in block.named_parameters()}
    xr = leaf(x)
    yk = at_codes(norm64(xr, p["norm"], 1e-6), kept_values(mc2, y))
    zk = at_codes(yk @ p["w1"].T + p["b1"], kept_values(mc2, z))
    want = xr + act(zk, "gelu")[0] @ p["w2"].T + p["b2"]
    want.backward(d.cpu().double())
    near(x.grad, xr.grad, "x")
    for k, v in block.named_parameters():
        near(v.grad, p[k].grad, k)


def test_kept_gradients_are_near_the_16_bit_ones(ff):
    """What 8 bits cost: codes are off by half a step at most, 1/254 of their group's largest value, which of 128 normal
    values is about 2.7 deviations; a uniform error of that step is 2.7 / 127 / sqrt(12) = 0.006 of a deviation, once
    for x and twice over for z (slope and activation, slopes of them below 1.2).  5 of these in the 2-norm."""
    torch.manual_seed(2)
    plain, block = ff.FeedForward(256, 1024), ff.FeedForward(256, 1024, keep8=True)
    block.load_state_dict(plain.state_dict())
    x = torch.randn((300, 256), device="cuda").bfloat16()
    d = torch.randn((300, 256), device="cuda").bfloat16()
    for b in (plain, block):
        b(x).backward(d)
    for (k, a), b in zip(plain.named_parameters(), block.parameters()):
        err = torch.linalg.vector_norm(a.grad.double() - b.grad.double()) / torch.linalg.vector_norm(a.grad.double())
        assert err <= 5 * 0.006, (k, float(err))


def test_kept_bytes(ff):
    """Kept between forward and backward: the residual stream and codes, not 16-bit activations."""
    x = torch.randn((1024, 256), device="cuda").bfloat16().requires_grad_()
    kept = {}
    for keep8 in (False, True):
        block = ff.FeedForward(256, 1024, keep8=keep8)
        own = {p.data_ptr() for p in block.parameters()} | {x.data_ptr()}
        sizes = {}

        def pack(t):
            if t.data_ptr() not in own:
                sizes[t.data_ptr()] = t.numel() * t.element_size()
            return t
        with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
            out = block(x)
        kept[keep8] = sum(sizes.values()) / 1024
        del out
    scales = 4 * (256 + 1024) // 128
    assert kept[True] <= 256 + 1024 + scales + 2 * 256 + 8  # codes, scales; s where it is not x, rstd
    assert kept[False] >= 2 * 256 + 4 * 1024


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("score", [0, 1])
def test_experts_with_a_router_train(ff, keep8, score):
    import comm_matmul_tensor_amd as mc2
    torch.manual_seed(3)
    kind = dict(groups=4, top_groups=2, group_top=2, renormalise=bool(score), scale=1.5)
    block = ff.ExpertsFeedForward(128, 200, experts=12, top=3, score=score, balance=True, keep8=keep8, **kind)
    block.bias.copy_(torch.linspace(-0.05, 0.05, 12))
    x = torch.randn((90, 128), device="cuda").bfloat16()
    x[5] = 0.0  # equal scores for all: the bias and the order decide
    x.requires_grad_()
    out, s = block(x)
    d = torch.randn((90, 128), device="cuda").bfloat16()
    (out.float() * d.float()).sum().backward()
    assert torch.equal(s, x)
    p = {k: leaf(v) for k, v in block.named_parameters()}
    xr = leaf(x)
    with torch.no_grad():  # the choice is the operator's of the module's own logits, tested elsewhere
        y = mc2.mc2_add_rms_norm(x, block.norm)[0]
        logits = mc2.mc2_linear_act(y, block.router)[0]
        ids = mc2.mc2_moe_route(logits, 3, block.bias, score=score, **kind)[0]
        assert torch.equal(ids.cpu(), ref.route(logits.cpu(), 3, block.bias.cpu(), ["softmax", "sigmoid"][score], groups=4,
                                                top_groups=2, group_top=2)[0])
        rows, row_map, off = mc2.mc2_moe_permute(y, ids, 12)
        z = mc2.mc2_linear_act(rows, block.w1, act=block.act, group_offsets=off, need_z=True)[1]
    ids, row_map = ids.cpu().long(), row_map.cpu().long()
    assert (ids >= 0).all()
    yr = norm64(xr, p["norm"], 1e-6)
    scores = ref.scores(yr @ p["router"].T, ["softmax", "sigmoid"][score]) if score else torch.softmax(yr @ p["router"].T, 1)
    w = scores.gather(1, ids)
    w = 1.5 * (w / w.sum(1, keepdim=True) if score else w)
    yk, zk = kept_values(mc2, rows), kept_values(mc2, z)
    want = 0
    for j in range(3):
        yj, m = yr, row_map[:, j]
        if keep8:
            yj = at_codes(yj, yk[m])
        zj = torch.einsum("th,tkh->tk", yj, p["w1"][ids[:, j]])
        if keep8:
            zj = at_codes(zj, zk[m])
        want = want + w[:, j:j + 1] * torch.einsum("tk,thk->th", act(zj, "silu")[0], p["w2"][ids[:, j]])
    (want * d.cpu().double()).sum().backward()
    near(x.grad, xr.grad, "x")
    for k, v in block.named_parameters():
        near(v.grad, p[k].grad, k)


def test_blocks_train_on_no_tokens(ff):
    moe = ff.ExpertsFeedForward(128, 64, experts=4, top=2, keep8=True, score=1, balance=True)
    dense = ff.FeedForward(128, 256, keep8=True)
    x = torch.empty((0, 128), dtype=torch.bfloat16).cuda().requires_grad_()
    out = dense(*moe(x))
    out.backward(torch.empty_like(out))
    assert x.grad.shape == (0, 128)
    for m in (moe, dense):
        for name, p in m.named_parameters():
            assert p.grad is not None and torch.count_nonzero(p.grad) == 0, name
    assert ff.Int8FeedForward(dense)(x.detach()).shape == (0, 128)
    assert ff.Int8ExpertsFeedForward(moe)(x.detach())[0].shape == (0, 128)


# ------------------------------------------------------------------ served in int8
def slack(x, w, xs, ws):
    """Largest change of x @ w^T where each factor moves by half its row's step."""
    return 0.5 * (xs @ w.abs().sum(1)[None] + (x.abs().sum(1)[:, None] + 0.5 * xs * x.shape[1]) @ ws.T)


def test_int8_feed_forward(ff):
    """Call by call the operators' own results; as a whole within what half a step in each factor can move."""
    import comm_matmul_tensor_amd as mc2
    torch.manual_seed(4)
    block = ff.FeedForward(256, 600)
    with torch.no_grad():
        block.b1.copy_(torch.linspace(-0.5, 0.5, 600))
    served = ff.Int8FeedForward(block)
    assert not list(served.parameters())
    for tokens in (1, 7, 64, 333):
        x = torch.randn((tokens, 256), device="cuda").bfloat16()
        r = torch.randn((tokens, 256), device="cuda").bfloat16()
        out = served(x, r)
        q, qs, s, _ = mc2.mc2_add_rms_norm(x, block.norm, r, out_dtype=torch.int8)
        w1, w1s = mc2.mc2_quant_rows(block.w1.detach())
        w2, w2s = mc2.mc2_quant_rows(block.w2.detach())
        a = mc2.mc2_linear_i8(q, qs, w1, w1s, block.b1.detach(), act=block.act)
        aq, aqs = mc2.mc2_quant_rows(a)
        assert torch.equal(out, mc2.mc2_linear_i8(aq, aqs, w2, w2s, block.b2.detach(), s))
        with torch.no_grad():
            full = block(x, r).cpu().double()
        f = lambda t: t.detach().cpu().double()
        y = norm64(f(x) + f(r), f(block.norm), 1e-6)
        e1 = 1.13 * slack(y, f(block.w1), f(qs), f(w1s)) + 4 * U["bf16"] * (1 + f(a).abs())
        e2 = slack(f(a), f(block.w2), f(aqs), f(w2s)) + e1 @ f(block.w2).abs().T
        assert ((f(out) - full).abs() <= 1.05 * e2 + 4 * U["bf16"] * (1 + full.abs())).all()
        # and in the 2-norm near it: the steps' errors do not add up in one direction
        assert torch.linalg.vector_norm(f(out) - full) <= 0.05 * torch.linalg.vector_norm(full - f(s))


@pytest.mark.parametrize("score", [None, 1])
def test_int8_experts(ff, score):
    import comm_matmul_tensor_amd as mc2
    torch.manual_seed(5)
    block = ff.ExpertsFeedForward(256, 320, experts=8, top=2, score=score, balance=score is not None)
    served = ff.Int8ExpertsFeedForward(block)
    for tokens in (1, 16, 200):
        x = torch.randn((tokens, 256), device="cuda").bfloat16()
        out, s = served(x)
        with torch.no_grad():
            y = mc2.mc2_add_rms_norm(x, block.norm)[0]
            ids, w = block.choose(y)
            full = block(x)[0].double()
        assert torch.equal(s, x)
        rows, row_map, off = mc2.mc2_moe_permute(y, ids, 8)
        w1, w1s = mc2.mc2_quant_rows(block.w1.detach())
        w2, w2s = mc2.mc2_quant_rows(block.w2.detach())
        a = mc2.mc2_linear_i8(*mc2.mc2_quant_rows(rows), w1, w1s, act=block.act, group_offsets=off)
        e = mc2.mc2_linear_i8(*mc2.mc2_quant_rows(a), w2, w2s, group_offsets=off)
        assert torch.equal(out, mc2.mc2_moe_unpermute(e, row_map, w))
        assert torch.linalg.vector_norm(out.double() - full) <= 0.05 * torch.linalg.vector_norm(full)


def test_a_decoding_step_in_a_graph(ff):
    """Experts and a dense block in int8 for a few tokens, captured, replayed on new ones with eager work between."""
    torch.manual_seed(6)
    moe = ff.Int8ExpertsFeedForward(ff.ExpertsFeedForward(256, 128, experts=8, top=2, score=1, groups=4, top_groups=2,
                                                          group_top=2, balance=True))
    dense = ff.Int8FeedForward(ff.FeedForward(256, 512))
    x = torch.randn((5, 256), device="cuda").bfloat16()
    dense(*moe(x))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dense(*moe(x))
    for seed in (7, 8, 9):
        torch.manual_seed(seed)
        x.copy_(torch.randn((5, 256), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dense(*moe(x)))


@pytest.mark.parametrize("score", [0, 1])
def test_a_training_step_in_a_graph(ff, score):
    """Forward and backward of a routed and a dense block that keep 8 bits, captured together while no eager graph of
    their parameters lives, replayed on new rows and gradients with eager steps between."""
    torch.manual_seed(8)
    moe = ff.ExpertsFeedForward(256, 128, experts=8, top=2, keep8=True, score=score, groups=4, top_groups=2, group_top=2,
                                renormalise=score == 1, balance=True)
    dense = ff.FeedForward(256, 384, keep8=True)
    leaves = [*moe.parameters(), *dense.parameters()]
    x = torch.randn((37, 256), device="cuda").bfloat16().requires_grad_()
    dout = torch.randn((37, 256), device="cuda").bfloat16()

    def step():
        out = dense(*moe(x))
        return out.detach(), *torch.autograd.grad(out, [x, *leaves], dout)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (9, 10, 11):
        torch.manual_seed(seed)
        with torch.no_grad():
            x.copy_(torch.randn((37, 256), device="cuda"))
            dout.copy_(torch.randn((37, 256), device="cuda"))
            moe.bias.copy_(torch.randn((8,), device="cuda") * 0.1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_state_moves_with_the_module(ff):
    torch.manual_seed(7)
    a = ff.Int8ExpertsFeedForward(ff.ExpertsFeedForward(128, 64, experts=4, top=2, score=0, balance=True))
    b = ff.Int8ExpertsFeedForward(ff.ExpertsFeedForward(128, 64, experts=4, top=2, score=0, balance=True))
    x = torch.randn((9, 128), device="cuda").bfloat16()
    assert not torch.equal(a(x)[0], b(x)[0])
    b.load_state_dict(a.state_dict())
    assert torch.equal(a(x)[0], b(x)[0])


@pytest.mark.parametrize("act_name", ["relu", "gelu", "gelu_tanh", "silu"])
def test_an_overflowed_pre_activation_keeps_its_neighbours(ff, act_name):
    """z past fp16's range is saved as -inf, whose activation and slope are 0.  It stays one among the codes, and its 128
    columns keep those of their finite values; the gradients are those of the formula at these values (near()'s
    bound, of the coarser type)."""
    import comm_matmul_tensor_amd as mc2
    from layer_ref import ACTS
    torch.manual_seed(12)
    code = ACTS.index(act_name)
    block = ff.FeedForward(192, 400, act=code, dtype=torch.float16, keep8=True)
    with torch.no_grad():
        block.b1.copy_(torch.linspace(-0.5, 0.5, 400))
        for col in (5, 130, 399):
            block.b1[col] = -65504.0
            block.w1[col].zero_()
            block.w1[col, 0] = -400.0  # -inf where the row's first value is 1, else finite
        block.b1[256:384] = -65504.0   # a group of nothing else
        block.w1[256:384].zero_()
        block.w1[256:384, 1] = -400.0
    x = torch.randn((77, 192), device="cuda").half()
    x[:, 0], x[:, 1] = 1.0, 1.0
    x[40:] = -x[40:].abs()             # these rows are finite
    x.requires_grad_()
    d = torch.randn((77, 192), device="cuda").half()
    out = block(x)
    assert torch.isfinite(out).all()
    out.backward(d)
    with torch.no_grad():
        y = mc2.mc2_add_rms_norm(x, block.norm)[0]
        z = mc2.mc2_linear_act(y, block.w1, block.b1, act=code, need_z=True)[1].cpu()
    low = z == -float("inf")
    assert low[:40, 5].all() and low[:40, 256:384].all() and not low[40:].any() and torch.isfinite(z[~low]).all()
    zk = ref.values(*ref.codes(torch.where(low, torch.zeros_like(z), z), 128), 128)
    zk[low] = -1e4
    p = {k: leaf(v) for k, v in block.named_parameters()}
    xr = leaf(x)
    yk = at_codes(norm64(xr, p["norm"], 1e-6), kept_values(mc2, y))
    zr = at_codes(yk @ p["w1"].T + p["b1"], zk)
    # (relu's slope at a value of 0, which many codes are, is 0; autograd's of the clamp in act() is 1)
    ar = torch.relu(zr) if act_name == "relu" else act(zr, act_name)[0]
    want = xr + ar @ p["w2"].T + p["b2"]
    want.backward(d.cpu().double())
    near(x.grad, xr.grad, "x")
    for k, v in block.named_parameters():
        near(v.grad, p[k].grad, k)


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("score", [None, 0, 1])
def test_a_token_without_a_usable_logit_is_nan(ff, score, keep8):
    """A NaN among a token's logits, or under a softmax one past fp16's range: its row is NaN whichever way the experts
    are chosen, trained or served in int8, and the other tokens' rows are what they are without it."""
    torch.manual_seed(11)
    kind = {} if score is None else dict(score=score, groups=4, top_groups=2, group_top=2, balance=True)
    block = ff.ExpertsFeedForward(128, 64, experts=8, top=2, dtype=torch.float16, keep8=keep8, **kind)
    x = torch.randn((21, 128), device="cuda").half()
    x[7] = 1.0  # its norm is a row of ones
    for case in ("nan", "inf"):
        with torch.no_grad():
            if case == "nan":
                block.router[3].copy_(torch.randn((128,), device="cuda") * 128 ** -0.5)
                x[7, 5] = float("nan")
            else:
                x[7, 5] = 1.0
                block.router[3].fill_(600.0)  # 128 * 600 is past 65504, a random row's sum is not
        others = [t for t in range(21) if t != 7]
        gone = case == "nan" or score != 1
        for module in (block, ff.Int8ExpertsFeedForward(block)):
            out, s = module(x)
            alone, _ = module(x[others].contiguous())
            assert torch.isnan(out[7]).all() if gone else torch.isfinite(out[7]).all(), (case, module)
            assert torch.equal(out[others], alone), (case, module)
        if gone:  # its gradients are NaN as well, the other tokens' are not
            v = x.detach().clone().requires_grad_()
            block(v)[0].float().sum().backward()
            assert torch.isnan(v.grad[7]).all() and torch.isfinite(v.grad[others]).all(), case


def test_a_frozen_block_keeps_nothing(ff):
    """With grad mode on, where nothing needs a gradient: the forward's bits, and no saved tensor."""
    torch.manual_seed(13)
    for block in (ff.FeedForward(128, 256, keep8=True), ff.ExpertsFeedForward(128, 64, experts=4, top=2, keep8=True)):
        x = torch.randn((33, 128), device="cuda").bfloat16()
        want = block(x)
        block.requires_grad_(False)
        saved = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t) or t, lambda t: t):
            out = block(x)
        out, want = (out, want) if isinstance(out, torch.Tensor) else (out[0], want[0])
        assert saved == [] and not out.requires_grad and torch.equal(out, want)


def test_kept_bytes_of_experts(ff):
    """Kept between forward and backward of an experts block per token: for each of its `top` rows codes and scales of
    h + hidden columns in place of 2 h + 4 hidden bytes, and in either case the experts' output (2 h); the normed
    rows that the router read (2 h), and small change: logits, ids, maps and weights, the residual stream."""
    h, hidden, top, experts, tokens = 256, 1024, 4, 8, 1024
    x = torch.randn((tokens, h), device="cuda").bfloat16().requires_grad_()
    kept = {}
    for keep8 in (False, True):
        block = ff.ExpertsFeedForward(h, hidden, experts, top, keep8=keep8, score=1)
        own = {p.data_ptr() for p in block.parameters()} | {x.data_ptr()}
        sizes = {}

        def pack(t):
            if t.data_ptr() not in own:
                sizes[t.data_ptr()] = t.numel() * t.element_size()
            return t
        with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
            out = block(x)
        kept[keep8] = sum(sizes.values()) / tokens
        del out
    # logits 2 each, ids, row_map and weights 4 each; rstd, and the ranges over all tokens
    small = 2 * experts + 12 * top + 8
    scales = 4 * (h + hidden) // 128
    assert top * (h + hidden + 2 * h) + 2 * h <= kept[True] <= top * (h + hidden + scales + 2 * h) + 2 * h + small + 2 * h
    assert kept[False] >= top * (2 * h + 4 * hidden + 2 * h) + 2 * h
