"""The RMS norm's rows at the ends of bf16's range."""

import pytest
import torch

from train_ref import BF16, DEV, F32, check_norm, rnd, within

pytestmark = pytest.mark.gpu

MOST, LEAST = float(torch.finfo(torch.bfloat16).max), 2.0 ** -133         # the least bf16 value that is not 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [8, 896, 4096, 8192, 32768])
def test_rows_of_the_largest_values(lib, dim, fmt):
    """Their squares leave f32's range, and so would squares 2^-70 of the rows, of wide ones.  (rstd is below f32's
    smallest normal value for the first row: 2^-149 is its step.)"""
    x = torch.sign(rnd(3, dim).float()) * MOST
    x[1] *= 2.0 ** -20
    x[2, 1:] = 1.0
    x = x.to(torch.bfloat16)
    w = rnd(dim, seed=2)
    y, s, rstd = lib.rms_norm(x, w, format=fmt, training=True)
    r64 = (x.double().square().mean(1) + 1e-6) ** -0.5
    within(rstd, r64, 64 * F32 * r64 + 2.0 ** -149, "rstd")
    if fmt == "bf16":
        want = x.double() * r64[:, None] * w.double()
        within(y, want, (BF16 + 2.0 ** -20) * want.abs() + 1e-39, "y")
    else:
        check_norm((y[0][1:], y[1][1:]), s[1:], None, x[1:], w)
        assert bool(y[1].isfinite().all()) and bool((y[0][0].float().abs().amax() == 448))
