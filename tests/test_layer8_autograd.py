"""The autograd functions of the router and of linears kept in 8 bits, on the CPU over torch stand-ins of the libmc2
calls (whose codes are the values themselves): what they save, pass on and return, and what they refuse."""
import pytest
import torch

import comm_matmul_tensor_amd.feed_forward as ff
from test_feed_forward_autograd import leaf, linear_act, linear_act_grad, silu, squares, total



def quant_rows(x, *, group):
    assert group == 128
    return x.detach().clone(), torch.ones((x.shape[0], 1), dtype=x.dtype)


def linear_act_grad_i8(dout, x, xs, w, z=None, zs=None, *, act, x_act=0, group_offsets=None, need_dx=True, need_dw=True,
                       need_dbias=False):
    assert (z is None) == (zs is None)
    return linear_act_grad(dout, silu(x) if x_act == ff.MC2_ACT_SILU else x, w, z, act=act, need_dx=need_dx,
                           need_dw=need_dw, need_dbias=need_dbias)


def moe_route(logits, top, bias=None, *, score, renormalise=True, scale=1.0):
    p = torch.softmax(logits, 1) if score == 0 else torch.sigmoid(logits)
    ids = (p if bias is None else p + bias).topk(top, dim=1).indices
    w = p.gather(1, ids)
    return ids.to(torch.int32), scale * (w / w.sum(1, keepdim=True) if renormalise else w)


def moe_route_grad(dweights, logits, ids, *, score, renormalise=True, scale=1.0):
    with torch.enable_grad():
        l = logits.detach().requires_grad_()
        p = torch.softmax(l, 1) if score == 0 else torch.sigmoid(l)
        w = p.gather(1, ids.long())
        w = scale * (w / w.sum(1, keepdim=True) if renormalise else w)
        return torch.autograd.grad((w * dweights).sum(), l)[0]


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    for fn in (linear_act, linear_act_grad_i8, quant_rows, moe_route, moe_route_grad):
        monkeypatch.setattr(ff, "mc2_" + fn.__name__, fn)


def calls():
    kept = lambda code: lambda x, w1, b1, w2, b2, r: ff.KeptLinearsFunction.apply(x, w1, b1, w2, b2, r, code, None)
    bare = lambda x, w1, w2: ff.KeptLinearsFunction.apply(x, w1, None, w2, None, None, ff.MC2_ACT_SILU, None)
    route = lambda bias, **kind: lambda l: ff.RouteFunction.apply(l, bias, 3, kind)[1]
    six = (leaf(3, 8), leaf(5, 8), leaf(5), leaf(8, 5), leaf(8), leaf(3, 8))
    return {
        "kept, silu": (kept(ff.MC2_ACT_SILU), six),
        "kept, no biases": (bare, (leaf(3, 8), leaf(5, 8), leaf(8, 5))),
        "route, softmax": (route(None, score=0), (leaf(4, 7),)),
        "route, sigmoid": (route(torch.linspace(0, 1e-3, 7).double(), score=1, renormalise=False, scale=2.5), (leaf(4, 7),)),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_first_derivatives(name):
    torch.manual_seed(1)
    fn, ts = calls()[name]
    assert torch.autograd.gradcheck(fn, ts)


@pytest.mark.parametrize("loss", [total, squares])
@pytest.mark.parametrize("name", sorted(calls()))
def test_second_derivatives_are_refused(name, loss):
    torch.manual_seed(2)
    fn, ts = calls()[name]
    grads = torch.autograd.grad(loss(fn(*ts)), ts, create_graph=True)
    for g, p in zip(grads, torch.autograd.grad(loss(fn(*ts)), ts)):
        assert torch.equal(g, p)
        with pytest.raises(RuntimeError, match="second derivatives"):
            (fn(*ts).sum() + g.square().sum()).backward(retain_graph=True)


def test_only_what_is_needed_is_computed(monkeypatch):
    """Frozen parameters: no gradient is asked for that nothing needs, and none of the first linear where all is frozen."""
    asked = []

    def spy(dout, x, xs, w, z=None, zs=None, **kw):
        asked.append((kw["need_dx"], kw["need_dw"], kw["need_dbias"]))
        return linear_act_grad_i8(dout, x, xs, w, z, zs, **kw)

    monkeypatch.setattr(ff, "mc2_linear_act_grad_i8", spy)
    for live, want in (((0,), [(True, False, False), (True, False, False)]), ((3, 4), [(False, True, True)]),
                       ((2,), [(True, False, False), (False, False, True)]), ((5,), [(False, False, False)])):
        ts = [t.detach().requires_grad_(i in live) for i, t in enumerate(calls()["kept, silu"][1])]
        asked.clear()
        ff.KeptLinearsFunction.apply(*ts, ff.MC2_ACT_SILU, None).sum().backward()
        assert asked == want, live
        assert all((t.grad is not None) == (i in live) for i, t in enumerate(ts))


def test_gradients_arrive_aligned(monkeypatch):
    seen = []
    for fn in (linear_act_grad_i8, moe_route_grad):
        def checked(*args, _fn=fn, **kwargs):
            seen.append(all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in args if isinstance(t, torch.Tensor)))
            return _fn(*args, **kwargs)
        monkeypatch.setattr(ff, "mc2_" + fn.__name__, checked)
    for name in calls():
        fn, ts = calls()[name]
        out = fn(*ts)
        wide = torch.randn((out.numel() + 1,), dtype=torch.float64)
        for grad in (wide[1:].view(out.shape), torch.ones(()).double().expand(out.shape)):
            torch.autograd.grad(out, ts, grad, retain_graph=True)
    assert seen and all(seen)


def test_a_score_is_needed_for_groups_and_balance():
    for kw in (dict(groups=2, top_groups=1), dict(balance=True), dict(scale=2.0), dict(renormalise=False)):
        with pytest.raises(ValueError, match="need a score"):
            ff.ExpertsFeedForward(8, 8, 4, 2, device="cpu", **kw)
    assert ff.ExpertsFeedForward(8, 8, 4, 2, device="cpu").bias is None
    block = ff.ExpertsFeedForward(8, 8, 4, 2, device="cpu", score=1, balance=True)
    assert block.bias.shape == (4,) and "bias" in block.state_dict()


def test_nothing_is_kept_where_nothing_needs_a_gradient(monkeypatch):
    """A frozen block on rows that need no gradient, evaluated with grad mode on: no codes, no pre-activation."""
    made = []

    def codes(x, *, group):
        made.append(x.shape)
        return quant_rows(x, group=group)

    wanted = []

    def linear(*args, need_z=False, **kw):
        wanted.append(need_z)
        return linear_act(*args, need_z=need_z, **kw)

    monkeypatch.setattr(ff, "mc2_quant_rows", codes)
    monkeypatch.setattr(ff, "mc2_linear_act", linear)
    ts = [t.detach() for t in calls()["kept, silu"][1]]
    out = ff.KeptLinearsFunction.apply(*ts, ff.MC2_ACT_SILU, None)
    assert not out.requires_grad and made == [] and wanted == [False, False]
    for live in range(6):
        made.clear()
        again = ff.KeptLinearsFunction.apply(*(t.clone().requires_grad_(i == live) for i, t in enumerate(ts)),
                                             ff.MC2_ACT_SILU, None)
        assert torch.equal(again, out) and len(made) == 2
