"""How near the loss's logits come to 64 bits, for rows of every kind.

With a vocabulary of one word lse is that word's logit.  The matrix units sum 16 products a step and cut what falls
below the running sum's last place: up to 2^-23 of it (or of the step's largest product) a step.  1024 features are
summed that way at most, 64 steps; the parts join in f32, each rounding up or down by 2^-24 of itself or of
the sum.  Six roundings of the result follow (the logit's scale, its own and back from units of ln 2)."""

import pytest
import torch

from train_ref import DEV, F32

pytestmark = pytest.mark.gpu

PART = 1024


def rows(kind, M, h, V, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    ru = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    W, x = rn(V, h) * h ** -0.5, 2 * rn(M, h)
    if kind == "pulled":
        x = x + 12 * ru(M, 1) * W[y] * (h / 1024) ** 0.5
    if kind == "one sign":
        W, x = ru(V, h) / h * 20, ru(M, h) + 0.5
    if kind == "sparse":                             # one in twenty, of one sign
        W, x = ru(V, h) / h * 20, (ru(M, h) + 0.5) * (ru(M, h) < 0.05) * 8
    if kind == "heavy":
        x, W = x * torch.exp(1.5 * rn(M, h)), W * torch.exp(rn(V, h)) * 0.2
    return x.to(torch.bfloat16), W.to(torch.bfloat16), y


def cuts(x, w):
    """(logits, how far they may be off): rows x of one word."""
    prod = (x.double() * w.double()).unflatten(1, (-1, 16))
    step = prod.sum(2)
    pad = -step.shape[1] % (PART // 16)
    run = torch.nn.functional.pad(step, (0, pad)).unflatten(1, (-1, PART // 16)).cumsum(2)
    parts = run[:, :, -1]
    z = parts.sum(1)
    cut = 2 * F32 * (run.abs().sum((1, 2)) + prod.abs().amax(2).sum(1))
    joins = F32 * (parts.abs() + parts.cumsum(1).abs()).sum(1) if parts.shape[1] > 1 else 0.0
    return z, cut + joins + 6 * F32 * z.abs()


@pytest.mark.parametrize("kind", ["normal", "pulled", "one sign", "sparse", "heavy"])
@pytest.mark.parametrize("h", [896, 4096, 32768])
def test_logits(lib, h, kind):
    x, W, _ = rows(kind, 512, h, 1)
    y = torch.zeros(512, dtype=torch.int64, device=DEV)
    z, off = cuts(x, W[0])
    for grad in (False, True):
        lse = lib.linear_cross_entropy(x, W, y, grad=grad)[2].double()
        err = lse - z
        assert bool((err.abs() <= off).all()), f"{float((err.abs() / off).max()):.2f} of what is allowed"
        if kind in ("one sign", "sparse"):           # sums of positive products only lose
            assert float((err / z).max()) <= 8 * F32 * (1 + h // PART) and bool((z > 0).all())
    assert lib.poll_status() == 0


@pytest.mark.parametrize("kind", ["normal", "pulled", "one sign", "sparse", "heavy"])
@pytest.mark.parametrize("h", [896, 4096])
def test_loss(lib, h, kind):
    """Half a last place a step is cut on average: 0.36 * 2^-23 of the running sum, which stands at half its
    end on average, over 64 steps 1.4e-6 of a logit that grows steadily, and 1.4e-6 of each part's
    reach where it wanders.  The loss takes the label's logit and the mean of the others by their weight: rms over
    the rows at most 1.5 times that of the two, and f32's own 2^-22 of lse."""
    M, V = 256, 5003
    x, W, y = rows(kind, M, h, V)
    xd, wd = x.double(), W.double()
    z = xd @ wd.T
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, y[:, None])[:, 0]
    # the reach of a logit's parts: the sum of their sizes
    reach = sum((xd[:, a:a + PART] @ wd[:, a:a + PART].T).abs() for a in range(0, h, PART))
    mean = (torch.softmax(z, 1) * reach).sum(1)
    limit = 1.5 * 1.4e-6 * (mean + reach.gather(1, y[:, None])[:, 0]) + 4 * F32 * lse.abs()
    for grad in (False, True):
        got = lib.linear_cross_entropy(x, W, y, grad=grad)
        rms = lambda t: float(t.double().square().mean().sqrt())  # noqa: E731
        print(h, kind, grad, "loss %.2e lse %.2e of themselves; loss %.2f of what is allowed" % (
            rms(got[1].double() - loss) / rms(loss), rms(got[2].double() - lse) / rms(lse), rms(got[1].double() - loss) / rms(limit)))
        assert rms(got[1].double() - loss) <= rms(limit)
        assert rms(got[2].double() - lse) <= rms(limit)
    assert lib.poll_status() == 0
