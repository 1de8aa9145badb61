"""Narrow rows by the ten thousand: a group of threads takes two rows at once where that leaves the GPU full."""

import pytest
import torch

from train_ref import DEV, check_norm, rnd

pytestmark = pytest.mark.gpu


def edge(dim):
    """Rows from which on two are taken at once, on this GPU: 8 blocks of 128 threads an SM, two rows a group."""
    group = next(t for t in (8, 16, 32) if dim <= 8 * t)
    return torch.cuda.get_device_properties(0).multi_processor_count * 8 * (128 // group) * 2


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [8, 64, 72, 128, 136, 256])
def test_around_the_edge(lib, dim, fmt):
    n = edge(dim)
    for tokens, add in ((n - 1, True), (n, False), (n, True), (n + 1, True), (n + 29, False), (2 * n + 17, True)):
        x, w = rnd(tokens, dim), rnd(dim, seed=2)
        r = rnd(tokens, dim, seed=3) if add else None
        y, s, rstd = lib.rms_norm(x, w, residual=r, offset=1.0, format=fmt, training=True)
        check_norm(y, s, rstd, x, w, r, offset=1.0)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("dim,heads", [(64, 14), (128, 3), (256, 5)])
def test_heads_of_a_packed_buffer(lib, dim, heads):
    tokens = edge(dim) // heads + 7
    packed, w = rnd(tokens, 3 * heads, dim), rnd(dim, seed=2)
    x, r = packed[:, heads:2 * heads], rnd(heads, tokens, dim, seed=3).transpose(0, 1)
    out = torch.full((tokens, heads, 2 * dim), float("nan"), dtype=torch.bfloat16, device=DEV)
    y, s, rstd = lib.rms_norm(x, w, residual=r, training=True, sum_out=out[..., dim:])
    check_norm(y, s, rstd, x, w, r)
    assert bool(out[..., :dim].isnan().all())
    y, s, rstd = lib.rms_norm(x, w, format="fp8", training=True)
    check_norm(y, s, rstd, x, w)


def test_in_place_and_rows_that_are_not_finite(lib):
    tokens = edge(128) + 3
    x, r, w = rnd(tokens, 128), rnd(tokens, 128, seed=3), rnd(128, seed=2)
    want = lib.rms_norm(x, w, residual=r)
    a, b = x.clone(), r.clone()
    y, s, _ = lib.rms_norm(a, w, residual=b, sum_out=b)
    assert torch.equal(y, want[0]) and torch.equal(b, want[1])
    bad = x.clone()
    rows = torch.tensor([0, 5, tokens // 2, tokens - 1], device=DEV)
    bad[rows, 7] = float("nan")
    y = lib.rms_norm(bad, w, residual=r)[0]
    keep = torch.ones(tokens, dtype=torch.bool, device=DEV)
    keep[rows] = False
    assert torch.equal(y[keep], want[0][keep]) and bool(y[rows].isnan().all())
