"""The norm under autograd over tensors of unlike layouts: one contiguous, another a slice."""

import pytest
import torch

LAYOUTS = {
    "whole": lambda b, t, d: torch.empty(b, t, d), "slice": lambda b, t, d: torch.empty(b, t + 1, d)[:, 1:],
    "turned": lambda b, t, d: torch.empty(t, b, d).transpose(0, 1), "packed": lambda b, t, d: torch.empty(b, t, 3, d)[:, :, 1],
    "odd": lambda b, t, d: torch.empty(b, t, d + 3)[..., :d], "spread": lambda b, t, d: torch.empty(b, 1, d).expand(b, t, d),
    "feature-major": lambda b, t, d: torch.empty(b, d, t).transpose(1, 2),
}
PAIRS = [(a, b) for a in LAYOUTS for b in (None, *LAYOUTS)]


def laid(t, layout, dtype=torch.bfloat16):
    """t's values in another layout."""
    u = LAYOUTS[layout](*t.shape)
    if layout == "spread":
        return t[:, :1].to(dtype).expand(u.shape)
    size = sum((n - 1) * s for n, s in zip(u.shape, u.stride())) + 1 + u.storage_offset()
    return torch.zeros(size, dtype=dtype, device=t.device).as_strided(u.shape, u.stride(), u.storage_offset()).copy_(t)


def plain(x, weight, *, residual=None, eps, offset, training):
    assert x.shape == (x if residual is None else residual).shape, "residual must have x's shape"
    assert x.dim() == 2 or (x.dim() == 3 and x.shape[1] <= 65535)
    assert all(t is None or (t.stride(-1) == 1 and not any(s % 8 for s in t.stride()[:-1])) for t in (x, residual))
    s = x if residual is None else x + residual
    return s * 2, s, s.float().sum(-1)


@pytest.mark.parametrize("x,residual", PAIRS)
def test_routing(monkeypatch, x, residual):
    """What reaches the library: one shape, and strides that it takes."""
    from rank_mlp_gb300 import autograd
    monkeypatch.setattr(autograd, "binding", type("B", (), {"rms_norm": staticmethod(plain)}))
    g = torch.Generator().manual_seed(0)
    a, b = (torch.randn(2, 5, 64, generator=g) for _ in range(2))
    a = laid(a, x)
    r = None if residual is None else laid(b, residual)
    out = autograd.lora_rms_norm(a, torch.ones(64, dtype=torch.bfloat16), r)
    s = a if r is None else a + r
    if r is None:
        assert torch.equal(out, 2 * s)
    else:
        assert torch.equal(out[0], 2 * s) and torch.equal(out[1], s) and out[1].shape == a.shape


def test_routing_of_other_ranks_and_long_sequences(monkeypatch):
    from rank_mlp_gb300 import autograd
    monkeypatch.setattr(autograd, "binding", type("B", (), {"rms_norm": staticmethod(plain)}))
    w = torch.ones(8, dtype=torch.bfloat16)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    for a, r in ((z(8), None), (z(3, 8), z(6, 8)[::2]), (z(2, 3, 4, 8), z(2, 3, 5, 8)[:, :, 1:]), (z(2, 3, 16)[..., 8:], z(6, 8)),
                 (z(2, 70001, 8)[:, 1:], None), (z(2, 70001, 8)[:, 1:], z(2, 70000, 8))):
        out = autograd.lora_rms_norm(a, w, r)
        assert (out if r is None else out[0]).shape == a.shape


@pytest.mark.gpu
@pytest.mark.parametrize("x,residual", PAIRS)
def test_gradients(lib, x, residual):
    """Those of contiguous tensors, bit for bit."""
    from rank_mlp_gb300.autograd import lora_rms_norm
    from train_ref import rnd
    a, b, w = rnd(2, 5, 64), rnd(2, 5, 64, seed=1), rnd(64, seed=2)
    dy, ds = rnd(2, 5, 64, seed=3), rnd(2, 5, 64, seed=4)
    got = []
    for flat in (False, True):
        p, q = laid(a, x), None if residual is None else laid(b, residual)
        leaves = [t.contiguous() if flat else t for t in (p, q) if t is not None] + [w.clone()]
        for t in leaves:
            t.requires_grad_()
        out = lora_rms_norm(leaves[0], leaves[-1], *leaves[1:-1])
        torch.autograd.backward([out] if residual is None else list(out), [dy] if residual is None else [laid(dy, "turned"), laid(ds, "slice")])
        got.append([out if residual is None else out[0]] + [t.grad for t in leaves])
    for u, v in zip(*got):
        assert torch.equal(u, v)
    assert lib.poll_status() == 0
