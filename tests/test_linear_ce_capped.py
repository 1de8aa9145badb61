"""Capped logits far below their cap: a tanh keeps the relative precision of its argument."""

import pytest
import torch

from train_ref import BF16, DEV, F32, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [0.5, 30.0, 1000.0, 1e6])
def test_small_logits(lib, cap):
    """One word: lse is its capped logit.  The logit loses 2^-23 of its running sum and largest product a step of 16
    features at most; the tanh and the roundings around it 24 units of 2^-24."""
    M, h = 2000, 64
    x = (rnd(M, h, dtype=torch.float32) * torch.exp(torch.linspace(-9, 3, M, device=DEV))[:, None]).to(torch.bfloat16)
    W = rnd(1, h, seed=1, scale=h ** -0.5)
    y = torch.zeros(M, dtype=torch.int64, device=DEV)
    prod = (x.double() * W.double()).unflatten(1, (-1, 16))
    run = prod.sum(2).cumsum(1)
    z = run[:, -1]
    off = 2 * F32 * (run.abs().sum(1) + prod.abs().amax(2).sum(1))
    want = cap * torch.tanh(z / cap)
    for grad in (False, True):
        lse = lib.linear_cross_entropy(x, W, y, softcap=cap, grad=grad)[2]
        over = (lse.double() - want).abs() / (off + 24 * F32 * want.abs())
        assert bool((over <= 1).all()), f"{float(over.max()):.1f} times what is allowed"
    assert lib.poll_status() == 0


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
@pytest.mark.parametrize("cap", [1000.0, 1e6])
def test_a_cap_far_away(lib, cap, smoothing):
    """Logits of a spread of two under it: the loss moves by theirs only, 1e-5 at 128 features (8 steps, 2^-23 of up
    to 20 each), and dx keeps its weights' rounding."""
    M, h, V = 130, 128, 3000
    x, W = 2 * rnd(M, h), rnd(V, h, seed=1, scale=h ** -0.5)
    y = torch.randint(0, V, (M,), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    v = (x.double() @ W.double().T).requires_grad_()
    z = cap * torch.tanh(v / cap)
    lse = torch.logsumexp(z, 1)
    loss = lse - (1 - smoothing) * z.gather(1, y[:, None])[:, 0] - smoothing * z.mean(1)
    dz, = torch.autograd.grad(loss.sum(), v)
    d64 = dz @ W.double()
    for grad in (False, True):
        _, got, l, dx = lib.linear_cross_entropy(x, W, y, softcap=cap, smoothing=smoothing, reduction="sum", grad=grad)
        slack = 1e-5 + 64 * F32 * lse.abs()
        assert bool(((got.double() - loss).abs() <= slack).all()) and bool(((l.double() - lse).abs() <= slack).all())
        if grad:
            assert bool(((dx.double() - d64).norm(dim=1) <= 3 * BF16 * d64.norm(dim=1)).all())
    assert lib.poll_status() == 0


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
@pytest.mark.parametrize("M,h,V", [(130, 64, 300), (40, 2056, 1000)])
def test_logits_at_the_cap(lib, M, h, V, smoothing):
    """Rows whose logits reach 2 to 8 times the cap: all slopes are small, the label's too, and dx keeps its relative
    precision.  A slope 4 e^(-2x) takes twice the error of its argument (16 times 2e-6 here) and of its
    exponential; weights their rounding, and with smoothing what moves to the label's row."""
    cap = 5.0
    g = torch.Generator(device=DEV).manual_seed(0)
    u = torch.randn(h, generator=g, device=DEV)
    u = u / u.norm()
    reach = torch.linspace(2.0, 8.0, M, device=DEV)[:, None] * cap
    W = (u + 0.2 * torch.randn(V, h, generator=g, device=DEV) * h ** -0.5).to(torch.bfloat16)
    x = (reach * u + 0.05 * torch.randn(M, h, generator=g, device=DEV)).to(torch.bfloat16)
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    w64 = W.double()
    a = x.double() @ w64.T / cap
    z = cap * torch.tanh(a)
    slope = torch.cosh(a) ** -2
    assert float(slope.max(1).values.min()) < 1e-4
    dz = (torch.softmax(z, 1) - smoothing / V) * slope
    at = y[:, None]
    dz.scatter_add_(1, at, -(1 - smoothing) * slope.gather(1, at))
    d64 = dz @ w64
    size = (dz.abs() @ w64.norm(dim=1)[:, None])[:, 0]
    dx = lib.linear_cross_entropy(x, W, y, softcap=cap, smoothing=smoothing, reduction="sum")[3]
    err = (dx.double() - d64).norm(dim=1)
    over = err / (BF16 * d64.norm(dim=1) + (3 * BF16 + 1e-4) * size)
    assert bool((over <= 1).all()), f"{float(over.max()):.1f} times what is allowed"
    assert lib.poll_status() == 0
