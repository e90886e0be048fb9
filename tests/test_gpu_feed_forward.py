"""The feed-forward modules end to end against torch autograd in 64 bits.

Every intermediate is rounded to 8 bits (U = 2^-8), of which a path through a
block passes fewer than 8; the outputs and gradients are sums in which these
errors do not add up in one direction.  The bound is 8 U of the result's
root mean square in the 2-norm.
"""
import pytest
import torch

from layer_ref import U, act

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ff():
    assert torch.cuda.is_available()
    import comm_matmul_tensor_amd.feed_forward as m
    return m


def near(got, ref, what):
    d = torch.linalg.vector_norm(got.detach().cpu().double() - ref.detach())
    assert d <= 8 * U["bf16"] * torch.linalg.vector_norm(ref.detach()), (what, float(d))


def leaf(t):
    return t.detach().cpu().double().requires_grad_()


def norm64(x, w, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def test_feed_forward_trains(ff):
    torch.manual_seed(1)
    block = ff.FeedForward(192, 520)
    x = torch.randn((77, 192), device="cuda").bfloat16().requires_grad_()
    r = torch.randn((77, 192), device="cuda").bfloat16().requires_grad_()
    out = block(block(x, r))
    d = torch.randn((77, 192), device="cuda").bfloat16()
    out.backward(d)
    p = {k: leaf(v) for k, v in block.named_parameters()}
    xr, rr = leaf(x), leaf(r)

    def ref(v):
        return v + act(norm64(v, p["norm"], 1e-6) @ p["w1"].T + p["b1"], "gelu")[0] @ p["w2"].T + p["b2"]

    want = ref(ref(xr + rr))
    want.backward(d.cpu().double())
    near(out, want, "out")
    near(x.grad, xr.grad, "x")
    near(r.grad, rr.grad, "residual")
    for k, v in block.named_parameters():
        near(v.grad, p[k].grad, k)


def test_experts_train(ff):
    torch.manual_seed(2)
    block = ff.ExpertsFeedForward(128, 200, experts=6, top=2)
    x = torch.randn((90, 128), device="cuda").bfloat16().requires_grad_()
    out, s = block(x)
    d = torch.randn((90, 128), device="cuda").bfloat16()
    (out.float() * d.float()).sum().backward()
    p = {k: leaf(v) for k, v in block.named_parameters()}
    xr = leaf(x)
    y = norm64(xr, p["norm"], 1e-6)
    score = y @ p["router"].T
    # the choice itself is the module's (a tie or a near one may go either way after rounding)
    with torch.no_grad():
        ys = ff.mc2_add_rms_norm(x, block.norm)[0]
        ids = ff.mc2_linear_act(ys, block.router)[0].float().topk(2, dim=-1).indices.cpu()
    w = torch.softmax(score.gather(1, ids), dim=-1)
    want = 0
    for j in range(2):
        a = act(torch.einsum("th,tkh->tk", y, p["w1"][ids[:, j]]), "silu")[0]
        want = want + w[:, j:j + 1] * torch.einsum("tk,thk->th", a, p["w2"][ids[:, j]])
    (want * d.cpu().double()).sum().backward()
    assert torch.equal(s, x)
    near(out, want, "out")
    near(x.grad, xr.grad, "x")
    for k, v in block.named_parameters():
        near(v.grad, p[k].grad, k)


def test_blocks_chain_and_decode(ff):
    """Experts, then a dense block whose norm adds the experts' output; a token alone gives what it gives in a batch."""
    torch.manual_seed(3)
    moe, dense = ff.ExpertsFeedForward(256, 128, experts=4, top=1), ff.FeedForward(256, 512)
    x = torch.randn((40, 256), device="cuda").bfloat16()
    with torch.no_grad():
        whole = dense(*moe(x))
        for t in (0, 17, 39):
            one = dense(*moe(x[t:t + 1].contiguous()))
            near(one, whole[t:t + 1].cpu().double(), f"token {t}")
