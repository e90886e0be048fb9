"""The tensor-parallel autograd functions on the CPU, over torch stand-ins of the libmc2 calls: gradients of
the group against the whole product's, and second derivatives refused."""
import pytest
import torch

import comm_matmul_tensor_amd.linear as lin

R = 2


def allgather_matmul(xs, w, *, x2_trans=False, gather_output=True, _bias=None):
    full = torch.cat(list(xs))
    out = full @ (w.t() if x2_trans else w)
    return out if _bias is None else out + _bias, full if gather_output else None


def matmul_reduce_scatter(x, w, recv, rank, *, x2_trans=False, _bias=None):
    part = x @ (w.t() if x2_trans else w)
    rows = part.shape[0] // R
    out = part[rank * rows:(rank + 1) * rows]
    for block in recv:
        out = out if block is None else out + block
    return out if _bias is None else out + _bias, part


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    monkeypatch.setattr(lin, "mc2_allgather_matmul", allgather_matmul)
    monkeypatch.setattr(lin, "mc2_matmul_reduce_scatter", matmul_reduce_scatter)
    monkeypatch.setattr(lin, "mc2_matmul_grad_input", lambda g, w: g @ w)
    monkeypatch.setattr(lin, "mc2_matmul_grad_weight", lambda g, x: g.t() @ x)
    monkeypatch.setattr(lin, "mc2_bias_grad", lambda g: g.sum(0))


def leaf(*shape):
    return torch.randn(shape, dtype=torch.float64).requires_grad_()


def column(*ts):
    return torch.cat(lin.AllGatherMatmulFunction.apply(R, True, *ts), dim=1)


def row(*ts):
    return torch.cat(lin.MatmulReduceScatterFunction.apply(R, True, *ts))


def cases():
    return [(column, [leaf(3, 5), leaf(3, 5), leaf(4, 5), leaf(4, 5), leaf(4), leaf(4)]),
            (row, [leaf(6, 5), leaf(6, 5), leaf(4, 5), leaf(4, 5), leaf(4)])]


@pytest.mark.parametrize("which", [0, 1])
def test_first_derivatives(which):
    torch.manual_seed(1)
    fn, ts = cases()[which]
    assert torch.autograd.gradcheck(fn, ts)


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("which", [0, 1])
def test_second_derivatives_are_refused(which, square):
    torch.manual_seed(2)
    fn, ts = cases()[which]
    loss = lambda: (fn(*ts).square() if square else fn(*ts)).sum()
    grads = torch.autograd.grad(loss(), ts, create_graph=True)
    for g, p in zip(grads, torch.autograd.grad(loss(), ts)):
        assert torch.equal(g, p) and not p.requires_grad
        with pytest.raises(RuntimeError, match="second derivatives"):
            (loss() + g.square().sum()).backward(retain_graph=True)
