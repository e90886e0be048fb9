"""Blocks whose outputs are parts of a concatenation: their gradients are views at odd addresses."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_blocks_inside_a_concatenation():
    from comm_matmul_tensor_amd.feed_forward import ExpertsFeedForward, FeedForward
    torch.manual_seed(5)
    h = 67  # 3 rows of it end off every 16-byte boundary
    dense, moe = FeedForward(h, 40), ExpertsFeedForward(h, 24, experts=3, top=2)
    x = torch.randn((5, h), device="cuda").bfloat16().requires_grad_()
    parts = [dense(x[:3].clone()), dense(x[3:].clone()), moe(x[:3].clone())[0], moe(x[3:].clone())[0]]
    d = torch.randn((10, h), device="cuda").bfloat16()
    leaves = [x, *dense.parameters(), *moe.parameters()]
    got = torch.autograd.grad(torch.cat(parts), leaves, d, retain_graph=True)
    want = torch.autograd.grad(parts, leaves, [d[a:b].clone() for a, b in ((0, 3), (3, 5), (5, 8), (8, 10))])
    for g, w in zip(got, want):
        assert torch.equal(g, w)
