"""64-bit forms of the norm, the loss and the clipping, with how far the kernels may be from them.

A result rounded to a type is off by half its step at most (bf16 2^-8 of the value, e4m3 2^-4, and
2^-10 of a row's scale below its smallest normal code).  Before that an f32 sum of n terms in a
tree of chains is off by at most (length of the longest chain + depth) * 2^-24 of the sum of its
terms' magnitudes; the bounds below take a count that covers the kernels' chains.
"""

import torch

DEV = "cuda:0"
BF16, E4M3, F32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24


def rnd(*shape, seed=0, scale=1.0, dtype=torch.bfloat16, dev=DEV):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(dev)


def within(got, want, slack, name=""):
    """|got - want| <= slack everywhere, NaN where want is NaN."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} for {tuple(want.shape)}"
    bad = ~(((got - want).abs() <= slack) | (got.isnan() & want.isnan()) | (got == want))
    if bool(bad.any()):
        i = int(bad.flatten().nonzero()[0])
        s = slack.expand(want.shape).flatten()[i] if isinstance(slack, torch.Tensor) else slack
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; first at {i}: {float(got.flatten()[i])} for "
                             f"{float(want.flatten()[i])}, may be off by {float(s):.3g}")


# ------------------------------------------------------------------ norm

def norm64(s, weight, eps, offset):
    """(y, rstd) of rows s, already rounded."""
    s = s.double()
    rstd = (s.square().mean(-1) + eps) ** -0.5
    return s * rstd.unsqueeze(-1) * (weight.double() + offset), rstd


def check_norm(y, s, rstd, x, weight, residual=None, eps=1e-6, offset=0.0):
    """s bit for bit; rstd within the sum's chain (32 products a thread, 10 steps of joining) and its root;
    y within its rounding, or its code's."""
    want_s = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    assert torch.equal(s.contiguous().view(torch.int16), want_s.contiguous().view(torch.int16))
    y64, r64 = norm64(want_s, weight, eps, offset)
    if rstd is not None:
        within(rstd, r64, 64 * F32 * r64, "rstd")
    if not isinstance(y, tuple):
        within(y, y64, (BF16 + 100 * F32) * y64.abs() + 1e-39, "y")
        return
    codes, scale = y
    top = y64.abs().amax(-1)
    assert codes.dtype == torch.float8_e4m3fn
    within(scale, (top / 448).clamp(min=2.0 ** -126), 100 * F32 * top / 448 + 1e-45, "scale")
    step = scale.double().unsqueeze(-1)
    within(codes.float().double() * step, y64, (E4M3 + 200 * F32) * y64.abs() + step * 2.0 ** -10, "codes")


def norm_grad64(dy, s, weight, rstd, offset, ds):
    """(dx, dw, size of dx's terms, size of dw's terms)."""
    dy, n, r = dy.double(), s.double() * rstd.double().unsqueeze(-1), rstd.double().unsqueeze(-1)
    g = dy * (weight.double() + offset)
    dot = (g * n).mean(-1, keepdim=True)
    dx = r * (g - n * dot)
    size = r * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True))
    if ds is not None:
        dx = dx + ds.double()
        size = size + ds.double().abs()
    return dx, (dy * n).flatten(0, -2).sum(0), size, (dy * n).abs().flatten(0, -2).sum(0)


def check_norm_grad(dx, dw, dy, s, weight, rstd, offset=0.0, ds=None):
    x64, w64, xs, wsz = norm_grad64(dy, s, weight, rstd, offset, ds)
    within(dx, x64, BF16 * x64.abs() + 100 * F32 * xs + 1e-39, "dx")
    if dw is not None:
        rows = s.numel() // s.shape[-1]
        within(dw, w64, BF16 * w64.abs() + (rows + 700) * F32 * wsz + 1e-39, "dweight")


# ------------------------------------------------------------------ loss

def ce64(x, W, labels, scale=1.0, softcap=0.0, smoothing=0.0, ignore_index=-100, reduction="mean"):
    """(total, loss, lse, dx, slack of loss, slack of dx) of the definition, and how far f32 logits of
    bf16 rows, f32 exponentials and bf16 weights may be from it."""
    V, h = W.shape
    seen = labels != ignore_index
    at = torch.where(seen, labels, 0)
    x64, w64 = x.double(), W.double()
    x64 = torch.where(seen[:, None], x64, 0.0)
    v = scale * (x64 @ w64.T)
    # the matrix units round their running sum once each 16 products (by up to a whole unit
    # of the last place), and 16 products as they join
    dv = abs(scale) * (h / 16 + 16) * 2 * F32 * 2 * (x64.abs() @ w64.abs().T) + 4 * F32 * v.abs()
    z = softcap * torch.tanh(v / softcap) if softcap else v
    # exponent: its argument's rounding (up to 128 in units of ln 2), the exponential's own 2^-22,
    # with a cap the tanh's few units of the last place of the cap itself
    dz = dv + 16 * F32 * z.abs() + 16 * F32 * softcap
    lse = torch.logsumexp(z, 1)
    slope = 1 - (z / softcap) ** 2 if softcap else torch.ones_like(z)
    p = torch.exp(z - lse[:, None])
    zy = z.gather(1, at[:, None])[:, 0]
    loss = lse - (1 - smoothing) * zy - smoothing * z.mean(1)
    worst = dz.amax(1)
    chain = (V / 128 + 64) * F32                       # a sum over V in slots of 128 columns
    off = 2 * worst + 40 * F32 * (lse.abs() + 64) + chain + smoothing * (2 * z.abs().mean(1) * (chain + 64 * F32) + worst)
    n = max(1, int(seen.sum())) if reduction == "mean" else 1
    g = torch.where(seen, scale / n, 0.0)[:, None]
    target = torch.full_like(z, smoothing / V).scatter_add(1, at[:, None], torch.full_like(zy, 1 - smoothing)[:, None])
    dx = (g * (p - target) * slope) @ w64
    # weights: rounded to bf16, moved by their logit's error, summed in steps of 16 over V, then again
    # over up to 32 ranges; the label's own is f32
    rel = BF16 + 2 * worst[:, None] + (V / 16 + 64) * 2 * F32 + 64 * F32
    terms = (p * slope).scatter(1, at[:, None], 0.0) @ w64.abs()
    py = p.gather(1, at[:, None])
    wy = w64[at].abs()
    sy = slope.gather(1, at[:, None])
    label = ((1 - py) * (2 * worst[:, None] + 1e-5) + smoothing * 1e-5) * wy * sy + 64 * F32 * wy * (1 - py)
    flat = smoothing / V * ((V / 300 + 400) * F32 + 1e-5) * w64.abs().sum(0)
    if softcap:                                        # slopes move with their logits
        move = 4 * (dz / softcap).amax(1, keepdim=True) + 16 * F32
        terms_s = (p + target).matmul(w64.abs())
        label = label + move * terms_s
        if smoothing:                                  # the smoothing's share is in the rounded weights
            label = label + rel * smoothing / V * w64.abs().sum(0)
    slack = BF16 * dx.abs() + g.abs() * (rel * terms + label + flat) + 1e-38
    keep = lambda t: torch.where(seen, t, 0.0)  # noqa: E731
    return keep(loss).sum() / n, keep(loss), keep(lse), dx, keep(off), slack


def check_ce(got, x, W, labels, **kw):
    total, loss, lse, dx = got
    t64, l64, s64, d64, off, slack = ce64(x, W, labels, **kw)
    within(loss, l64, off + 4 * F32 * l64.abs(), "loss")
    within(lse, s64, off + 4 * F32 * s64.abs(), "lse")
    n = max(1, int((labels != kw.get("ignore_index", -100)).sum())) if kw.get("reduction", "mean") == "mean" else 1
    within(total, t64, (off.sum() + 4 * F32 * l64.abs().sum()) / n + 4 * F32 * t64.abs(), "total")
    if dx is not None:
        within(dx, d64, slack, "dx")
