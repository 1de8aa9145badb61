"""The loss over more tokens than a block counts by itself: their labels are packed by a launch of their own."""

import pytest
import torch

from train_ref import DEV, ce64, rnd, within

pytestmark = pytest.mark.gpu

EDGE = 16384


def problem(M, h, V, hide, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    W = (torch.randn(V, h, generator=g, device=DEV) * h ** -0.5).to(torch.bfloat16)
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    x = (2 * torch.randn(M, h, generator=g, device=DEV) + 6 * W[y].float()).to(torch.bfloat16)
    y[torch.rand(M, generator=g, device=DEV) < hide] = -100
    return x, W, y


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("M", [EDGE, EDGE + 1, 20003, 3 * EDGE + 5])
def test_against_smaller_calls(lib, M, grad):
    """A token's loss, lse and gradient do not depend on the tokens around it (rows of one tile or another take
    the same sums), but for the order of the k-ranges' sums of dx."""
    x, W, y = problem(M, 64, 700, 0.3, seed=M)
    total, loss, lse, dx = lib.linear_cross_entropy(x, W, y, reduction="sum", grad=grad)
    for a in range(0, M, 5000):
        part = slice(a, a + 5000)
        _, l, s, d = lib.linear_cross_entropy(x[part], W, y[part], reduction="sum", grad=grad)
        assert torch.equal(loss[part], l) and torch.equal(lse[part], s)
        if grad:
            _, _, _, d64, _, slack = ce64(x[part], W, y[part], reduction="sum")
            within(dx[part], d64, slack, "dx")
            within(d, d64, slack, "dx")
    assert abs(float(total) - float(loss.double().sum())) <= 1e-6 * float(loss.double().sum())
    hidden = y == -100
    assert not bool(loss[hidden].any()) and not bool(lse[hidden].any()) and bool((loss[~hidden] > 0).all())
    assert lib.poll_status() == 0


@pytest.mark.parametrize("M", [EDGE, EDGE + 1, 20003])
def test_labels_outside_the_vocabulary(lib, M):
    """Reported, and taken as no label: in the first and the last places, and about the scan's turns of 4096."""
    x, W, y = problem(M, 64, 700, 0.3)
    at = torch.tensor([0, 1, 4095, 4096, 8191, EDGE - 1, M - 1], device=DEV)
    z = y.clone()
    z[at] = torch.tensor([700, -1, 1 << 40, -(1 << 40), 701, -5, 1 << 33], device=DEV)
    got = lib.linear_cross_entropy(x, W, z)
    assert lib.poll_status() == 7
    y[at] = -100
    for a, b in zip(got, lib.linear_cross_entropy(x, W, y)):
        assert torch.equal(a, b)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("seen", [0, 1, 20002])
def test_one_label_or_none(lib, seen):
    M = 20003
    x, W, y = problem(M, 64, 700, 0.0)
    keep = int(y[seen])
    y[:] = -100
    if seen:
        y[seen] = keep
    total, loss, lse, dx = lib.linear_cross_entropy(x, W, y)
    assert int((loss != 0).sum()) == int((dx != 0).any(1).sum()) == (1 if seen else 0)
    one = lib.linear_cross_entropy(x[seen:seen + 1], W, y[seen:seen + 1])
    assert torch.equal(total, one[0]) and torch.equal(loss[seen:seen + 1], one[1])
    assert lib.poll_status() == 0
