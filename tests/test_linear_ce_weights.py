"""The gradient's weights of a head whose rows share a direction or are alike: what bf16 takes off or adds to
each weight may not add up along what the rows have in common.

With weights w_v (1 + d_v), |d_v| <= 2^-8, whose sum is made that of the w_v again, the error of a row of dx is
sum_v (d_v - D) w_v W_v, D = sum d_v w_v / sum w_v.  Its terms' factors sum to zero, so W_v may be replaced by
W_v - U with the same U throughout: the bound below has the rows' distances from their weighted mean, not
their lengths."""

import pytest
import torch

from train_ref import BF16, DEV, F32

pytestmark = pytest.mark.gpu

M, H, V = 200, 256, 4096


def problem(head, gap, seed=0):
    """A competing word beside the label: `gap` above it for the first row, up to 2 more for the last."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    y = torch.randperm(V, generator=g, device=DEV)[:2 * M]
    y, other = y[:M], y[M:]
    W = r(V, H) * H ** -0.5
    if "near" in head:
        W[other] = W[y] + 0.1 * r(M, H) * H ** -0.5
    own = W.clone()
    if "common" in head:
        W = W + 5.0 * r(1, H) * H ** -0.5
    W = W.to(torch.bfloat16)
    # two equations for x: 14 on the label's row, the gap along the rows' difference
    d = own[other] - own[y]
    x = 0.5 * r(M, H)
    want = torch.stack([torch.full((M,), 14.0, device=DEV), gap + torch.linspace(-1, 2, M, device=DEV)], 1)
    A = torch.stack([own[y], d], 1)                                          # [M, 2, H]
    rest = want - torch.einsum("mkh,mh->mk", A, x)
    x = x + torch.einsum("mkh,mk->mh", A, torch.linalg.solve(A @ A.transpose(1, 2), rest))
    return x.to(torch.bfloat16), W, y


def rows64(x, W, y, scale=1.0, softcap=0.0, smoothing=0.0):
    """(dx, bound of each row's error)."""
    w64 = W.double()
    v = scale * (x.double() @ w64.T)
    z = softcap * torch.tanh(v / softcap) if softcap else v
    p = torch.softmax(z, 1)
    slope = 1 - (z / softcap) ** 2 if softcap else torch.ones_like(z)
    flat = torch.full_like(z, smoothing / V)
    dz = (p - flat) * slope
    at = y[:, None]
    dz.scatter_add_(1, at, -(1 - smoothing) * slope.gather(1, at))
    dx = scale * (dz @ w64)
    # what is rounded: all but the label's, with the smoothing's part where there is a cap too
    signed = bool(softcap and smoothing)
    w = ((p - flat) * slope if signed else p * slope).scatter(1, at, 0.0)
    mean = (w @ w64) / w.sum(1, keepdim=True)
    far = lambda u: (w64.square().sum(1) - 2 * u @ w64.T + u.square().sum(1, keepdim=True)).clamp(min=0).sqrt()  # noqa: E731
    away = far(mean)
    if signed:                                       # (the label's row takes the difference where weights cancel)
        away = torch.maximum(away, far(w64[y]))
    spread = (w.abs() * away).sum(1)
    # logits move by 2e-6 of the largest at this h and 2^-22 (their exponentials); with a cap by its last
    # places; the matrix units sum V / 16 steps, up to 2^-23 of the sum each
    worst = 4e-6 * v.abs().amax(1) + 4 * F32 + 32 * F32 * softcap
    size = (w.abs() * w64.norm(dim=1)).sum(1)
    steps = (V / 16 + 64) * 2 * F32
    d = dx.norm(dim=1)
    slack = abs(scale) * ((3 if signed else 2) * BF16 + 2 * worst) * spread + (BF16 + 4 * worst) * d
    slack = slack + abs(scale) * (steps + 16 * F32) * size
    if smoothing:                                    # the flat part: f32 sums of V rows, and slopes that move
        slack = slack + abs(scale) * smoothing * ((V + 400) * F32 + 4 * worst) * w64.norm(dim=1).mean()
    if softcap:
        slack = slack + 4 * abs(scale) * worst / softcap * (size + w64[y].norm(dim=1) * (1 - p.gather(1, at)[:, 0]))
    return dx, slack


@pytest.mark.parametrize("kw", [dict(), dict(smoothing=0.1), dict(softcap=30.0), dict(softcap=30.0, smoothing=0.1), dict(scale=0.5)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()) or "plain")
@pytest.mark.parametrize("gap", [0.0, 4.0])
@pytest.mark.parametrize("head", ["independent", "common", "near", "near common"])
def test_rows_that_share_a_direction(lib, head, gap, kw):
    x, W, y = problem(head, gap)
    d64, slack = rows64(x, W, y, **kw)
    dx = lib.linear_cross_entropy(x, W, y, reduction="sum", **kw)[3]
    err = (dx.double() - d64).norm(dim=1)
    over = err / slack
    assert bool((over <= 1).all()), f"{int((over > 1).sum())} rows, {float(over.max()):.1f} times what is allowed"
    assert lib.poll_status() == 0


@pytest.mark.parametrize("head", ["common", "near common"])
def test_a_piece_that_is_taken_again(lib, head):
    """One label far below its row's largest logit: the whole piece's weights come from the second try."""
    x, W, y = problem(head, 2.0)
    far = torch.randn(H, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    x[17] = (400.0 * torch.sign(far)).to(torch.bfloat16)
    y[17] = int((x[17].double() @ W.double().T).argmin())
    z = x.double() @ W.double().T
    assert float(z[17].max() - z[17, y[17]]) > 110
    d64, slack = rows64(x, W, y)
    dx = lib.linear_cross_entropy(x, W, y, reduction="sum")[3]
    assert bool(((dx.double() - d64).norm(dim=1) <= slack).all())
    assert lib.poll_status() == 0


def test_a_piece_with_a_cap_that_is_taken_again(lib):
    """The same with a cap above the distance: the weights' own sums come after the row's factors."""
    x, W, y = problem("near common", 2.0)
    far = torch.randn(H, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    x[17] = (30.0 * torch.sign(far)).to(torch.bfloat16)
    kw = dict(softcap=300.0)
    z = 300.0 * torch.tanh(x[17].double() @ W.double().T / 300.0)
    y[17] = int(z.argmin())
    assert float(z.max() - z.min()) > 110
    d64, slack = rows64(x, W, y, **kw)
    dx = lib.linear_cross_entropy(x, W, y, reduction="sum", **kw)[3]
    assert bool(((dx.double() - d64).norm(dim=1) <= slack).all())
    assert lib.poll_status() == 0


@pytest.mark.parametrize("M,h", [(64, 128), (4096, 896), (2400, 2056)])
def test_a_common_direction_over_a_long_vocabulary(lib, M, h):
    """No word stands out, so the product with the head grows steadily along the common direction, over 8192 steps.
    4096 features are summed at a time, 256 steps of up to 2^-23 of the sum each: 2^-16 of half the part's end on average,
    whichever the rows; the parts join in f32.  Many rows fill whole waves of tiles, few are cut into ranges."""
    V, n = 131072, 48
    g = torch.Generator(device=DEV).manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    common = 5.0 * r(1, h) * h ** -0.5
    W = (r(V, h) * h ** -0.5 + common).to(torch.bfloat16)
    x = 1.5 * r(M, h)
    x = (x - (x @ common.T) * common / common.square().sum()).to(torch.bfloat16)
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    dx = lib.linear_cross_entropy(x, W, y, reduction="sum")[3][:n].double()
    w64 = W.double()
    p = torch.softmax(x[:n].double() @ w64.T, 1)
    p[torch.arange(n), y[:n]] -= 1
    d64 = p @ w64
    size = w64.norm(dim=1).mean()
    slack = (BF16 + 2e-5) * d64.norm(dim=1) + (2.0 ** -17 + 64 * F32) * size + BF16 * 4 * V ** -0.5 * size
    assert bool(((dx - d64).norm(dim=1) <= slack).all())
    along = ((dx - d64) @ (common[0] / common.norm()).double()).abs()
    # the output's rounding along one direction: 2^-8 of a feature, of unlike signs
    limit = 4 * BF16 * (d64.square() * (common[0] / common.norm()).double().square()).sum(1).sqrt() + (2.0 ** -17 + 64 * F32) * size
    assert bool((along <= limit).all()), f"{float((along / limit).max()):.2f}"
    assert lib.poll_status() == 0


@pytest.mark.parametrize("smoothing", [0.1, 0.6])
@pytest.mark.parametrize("V", [3, 300, 5003])
def test_capped_and_smoothed_weights_of_one_size(lib, V, smoothing):
    """Logits near zero: all weights but the label's are alike and so is their rounding, which their sum's factor takes
    away.  What is left is the output's rounding, weights that differ by their logits' 0.1 or less and so in
    a few of their 2^-8 steps, and 1e-5 of the terms."""
    M, h, n = 200, 64, 1.0
    g = torch.Generator(device=DEV).manual_seed(V)
    W = (torch.randn(V, h, generator=g, device=DEV) * h ** -0.5).to(torch.bfloat16)
    x = (0.001 * torch.randn(M, h, generator=g, device=DEV)).to(torch.bfloat16)
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    w64 = W.double()
    z = 30.0 * torch.tanh(x.double() @ w64.T / 30.0)
    slope = 1 - (z / 30.0) ** 2
    dz = (torch.softmax(z, 1) - smoothing / V) * slope
    dz.scatter_add_(1, y[:, None], -(1 - smoothing) * slope.gather(1, y[:, None]))
    d64 = dz @ w64
    dx = lib.linear_cross_entropy(x, W, y, softcap=30.0, smoothing=smoothing, reduction="sum")[3]
    size = (1 - smoothing) * w64.norm(dim=1).mean()
    # weights (1 - smoothing) / V that logits of 0.005 and less put into at most two neighbouring steps: independent of
    # the rows of W, so their errors add up like sqrt(V) of 2^-8 / V
    slack = BF16 * d64.norm(dim=1) + size * (BF16 * V ** -0.5 * 3 + 2e-5)
    assert bool(((dx.double() - d64).norm(dim=1) <= slack).all())
    elem = BF16 * d64.abs() + size * (BF16 * V ** -0.5 * 3 + 2e-5)
    assert bool(((dx.double() - d64).abs() <= elem).all())
