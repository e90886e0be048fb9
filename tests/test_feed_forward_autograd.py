"""The autograd functions of comm_matmul_tensor_amd.feed_forward on the CPU, over torch stand-ins of the
libmc2 calls: what they save, pass on and return, and what they refuse."""
import pytest
import torch

import comm_matmul_tensor_amd.feed_forward as ff

EPS = 1e-6


def silu(z):
    return z * torch.sigmoid(z)


def linear_act(x, w, bias=None, residual=None, *, act, group_offsets=None, need_z=False):
    z = x @ w.t() if bias is None else x @ w.t() + bias
    out = silu(z) if act == ff.MC2_ACT_SILU else z
    return out if residual is None else out + residual, z if need_z else None


def linear_act_grad(dout, x, w, z=None, *, act, group_offsets=None, need_dx=True, need_dw=True, need_dbias=False):
    p = None if z is None else torch.sigmoid(z)
    dz = dout if z is None else dout * p * (1 + z * (1 - p))
    return dz @ w if need_dx else None, dz.t() @ x if need_dw else None, dz.sum(0) if need_dbias else None


def add_rms_norm(x, weight, residual=None, *, eps, need_rstd=False):
    s = x if residual is None else x + residual
    rstd = torch.rsqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * weight, None, s, rstd


def add_rms_norm_grad(dout, s, weight, rstd, dsum=None):
    g, r = dout * weight, rstd[:, None]
    dx = r * (g - s * r * r * (g * s).mean(1, keepdim=True))
    return dx if dsum is None else dx + dsum, (dout * s * r).sum(0)


def moe_permute(x, ids, experts):
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    row_map = torch.empty_like(flat)
    row_map[order] = torch.arange(flat.numel(), dtype=flat.dtype)
    return x[order // ids.shape[1]], row_map.view(ids.shape), torch.zeros((experts + 1,), dtype=torch.int32)


def moe_unpermute(y, row_map, weights=None):
    rows = y[row_map.long()]
    return rows.sum(1) if weights is None else (rows * weights[:, :, None]).sum(1)


def moe_unpermute_grad(dout, y, row_map, weights=None, *, need_dweights=True):
    dy = torch.zeros_like(y)
    w = torch.ones(row_map.shape, dtype=y.dtype) if weights is None else weights
    dy[row_map.long().reshape(-1)] = (dout[:, None] * w[:, :, None]).reshape(-1, y.shape[1])
    return dy, (y[row_map.long()] * dout[:, None]).sum(2) if need_dweights else None


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    for fn in (linear_act, linear_act_grad, add_rms_norm, add_rms_norm_grad, moe_permute, moe_unpermute,
               moe_unpermute_grad):
        monkeypatch.setattr(ff, "mc2_" + fn.__name__, fn)


def leaf(*shape):
    return torch.randn(shape, dtype=torch.float64).requires_grad_()


def calls():
    """(function of tensors, its tensors) of every autograd function, with and without what is optional."""
    ids = torch.tensor([[1, 0], [2, 1], [0, 2]], dtype=torch.int32)
    row_map = moe_permute(torch.zeros((3, 1)), ids, 3)[1]
    norm = lambda x, r, w: ff.AddRMSNormFunction.apply(x, r, w, EPS)
    linear = lambda act: lambda x, w, b, r: ff.LinearActFunction.apply(x, w, b, r, act, None)
    return {
        "norm": (norm, (leaf(3, 8), leaf(3, 8), leaf(8))),
        "norm, no residual": (lambda x, w: norm(x, None, w), (leaf(3, 8), leaf(8))),
        "linear, silu": (linear(ff.MC2_ACT_SILU), (leaf(3, 8), leaf(5, 8), leaf(5), leaf(3, 5))),
        "linear alone": (lambda x, w: linear(ff.MC2_ACT_NONE)(x, w, None, None), (leaf(3, 8), leaf(5, 8))),
        "permute": (lambda x: ff.PermuteFunction.apply(x, ids, 3)[0], (leaf(3, 8),)),
        "unpermute": (lambda y, w: ff.UnpermuteFunction.apply(y, row_map, w), (leaf(6, 8), leaf(3, 2))),
        "unpermute, no weights": (lambda y: ff.UnpermuteFunction.apply(y, row_map, None), (leaf(6, 8),)),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_first_derivatives(name):
    torch.manual_seed(1)
    fn, ts = calls()[name]
    assert torch.autograd.gradcheck(fn, ts)


def total(out):
    return sum(o.sum() for o in (out if isinstance(out, tuple) else (out,)))


def squares(out):
    return total(tuple(o.square() for o in (out if isinstance(out, tuple) else (out,))))


@pytest.mark.parametrize("loss", [total, squares])
@pytest.mark.parametrize("name", sorted(calls()))
def test_second_derivatives_are_refused(name, loss):
    """Terms of a second derivative are never dropped: the backward through a gradient raises."""
    torch.manual_seed(2)
    fn, ts = calls()[name]
    grads = torch.autograd.grad(loss(fn(*ts)), ts, create_graph=True)
    plain = torch.autograd.grad(loss(fn(*ts)), ts)
    for g, p in zip(grads, plain):
        assert torch.equal(g, p) and not p.requires_grad  # the gradients themselves are as ever
    for g in grads:
        with pytest.raises(RuntimeError, match="second derivatives"):
            (fn(*ts)[0].sum() + g.square().sum()).backward(retain_graph=True)



def aligned(t):
    return t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0)


@pytest.mark.parametrize("name", sorted(calls()))
def test_gradients_arrive_aligned(name, monkeypatch):
    """A gradient may come in as a view at any address, as of a part of a concatenation: the library's calls get it
    contiguous and 16-byte aligned, which they require."""
    torch.manual_seed(4)
    seen = []
    for fn in (linear_act_grad, add_rms_norm_grad, moe_unpermute_grad, moe_unpermute):
        def checked(*args, _fn=fn, **kwargs):
            seen.append(all(aligned(a) for a in args if isinstance(a, torch.Tensor)))
            return _fn(*args, **kwargs)
        monkeypatch.setattr(ff, "mc2_" + fn.__name__, checked)
    fn, ts = calls()[name]
    outs = fn(*ts)
    for out in outs if isinstance(outs, tuple) else (outs,):
        wide = torch.randn((out.numel() + 1,), dtype=torch.float64)
        for grad in (wide[1:].view(out.shape), wide[1:].view(out.shape).t().contiguous().t(), torch.ones(()).double().expand(out.shape)):
            got = torch.autograd.grad(out, ts, grad, retain_graph=True, allow_unused=True)
            want = torch.autograd.grad(out, ts, grad.contiguous().clone(), retain_graph=True, allow_unused=True)
            for g, p in zip(got, want):
                assert (g is None) == (p is None) and (g is None or torch.equal(g, p))
    assert all(seen)
