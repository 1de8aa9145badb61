"""The loss under autograd: what reaches tokens that have no part in it."""

import pytest
import torch

from train_ref import DEV, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_gradients_of_unlabelled_tokens_losses_are_not_used(lib, bad):
    """A mean over weights that are zero where there is no label divides by zero there; the tokens' rows stay 0."""
    from rank_mlp_gb300.autograd import lora_linear_cross_entropy
    x, W = rnd(2, 30, 64), rnd(100, 64, seed=1, scale=0.1)
    y = torch.randint(0, 100, (2, 30), device=DEV)
    y[0, ::3] = -100
    y[1, 5:] = -100
    g = rnd(2, 30, seed=2, dtype=torch.float32)
    got = []
    for fill in (0.0, bad):
        leaf = x.clone().requires_grad_()
        lora_linear_cross_entropy(leaf, W, y, reduction="none").backward(torch.where(y == -100, fill, g))
        got.append(leaf.grad)
    leaf, own = x.clone().requires_grad_(), y.clone()
    loss = lora_linear_cross_entropy(leaf, W, own, reduction="none")
    own.fill_(7)                                     # the labels' buffer is filled again before the backward
    loss.backward(torch.where(y == -100, bad, g))
    assert torch.equal(leaf.grad, got[0])
    assert torch.equal(*got) and not bool(got[0][y == -100].any()) and bool(got[0][y != -100].any(1).all())
    assert lib.poll_status() == 0
