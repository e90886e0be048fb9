"""The gradient of the experts' rows where there is nothing to write: no rows, no tokens (a rank that got none)."""
import ctypes

import pytest
import torch

import comm_matmul_tensor_amd as mc2

A, NULL, I = ctypes.c_void_p(0x10000), None, ctypes.c_int64
OK, ERR_NULL, BF16 = 0, 1, 2


def grad(t, rows, dout=A, y=A, m=A, dy=NULL, dw=NULL):
    return ctypes.CDLL(mc2.LIB_PATH).mc2_moe_unpermute_grad(dout, y, m, NULL, I(t), I(2), I(128), I(rows), BF16, dy, dw,
                                                            NULL)


def test_nothing_to_write_is_a_valid_call():
    """Empty tensors have NULL addresses: such a call returns before any device work."""
    assert grad(0, 0, dout=NULL, y=NULL, m=NULL) == OK
    assert grad(0, 0, dout=NULL, y=NULL, m=NULL, dw=A) == OK
    assert grad(5, 0, y=NULL) == OK  # all choices dropped, dweights not wanted


def test_outputs_are_still_required_where_there_are_rows():
    assert grad(5, 10) == ERR_NULL
    assert grad(0, 10, dout=NULL, m=NULL) == ERR_NULL
    assert grad(5, 0, dout=NULL, y=NULL) == ERR_NULL and grad(5, 0, m=NULL, y=NULL) == ERR_NULL


@pytest.mark.gpu
def test_gradients_of_no_rows():
    empty, none = torch.empty((0, 16), dtype=torch.bfloat16).cuda(), torch.empty((0, 2), dtype=torch.int32).cuda()
    dy, dw = mc2.mc2_moe_unpermute_grad(empty, empty, none)
    assert dy.shape == (0, 16) and dw.shape == (0, 2)
    dy, dw = mc2.mc2_moe_unpermute_grad(empty, empty, none, need_dweights=False)
    assert dy.shape == (0, 16) and dw is None
    dout, dropped = torch.ones((5, 16), dtype=torch.bfloat16).cuda(), torch.full((5, 2), -1, dtype=torch.int32).cuda()
    dy, dw = mc2.mc2_moe_unpermute_grad(dout, empty, dropped)
    assert dy.shape == (0, 16) and dw.shape == (5, 2) and torch.count_nonzero(dw) == 0
    dy, _ = mc2.mc2_moe_unpermute_grad(dout, empty, dropped, need_dweights=False)
    assert dy.shape == (0, 16)


@pytest.mark.gpu
def test_blocks_train_on_no_tokens():
    from comm_matmul_tensor_amd.feed_forward import ExpertsFeedForward, FeedForward
    moe, dense = ExpertsFeedForward(128, 64, experts=4, top=2), FeedForward(128, 256)
    x = torch.empty((0, 128), dtype=torch.bfloat16).cuda().requires_grad_()
    out = dense(*moe(x))
    assert out.shape == (0, 128)
    out.backward(torch.empty_like(out))
    assert x.grad.shape == (0, 128)
    for m in (moe, dense):
        for name, p in m.named_parameters():
            assert p.grad is not None and torch.count_nonzero(p.grad) == 0, name
