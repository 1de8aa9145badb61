"""The few-row kernel's softmax weights over a bf16 cache carry 16 bits of significand: where
V's rows cancel, the result keeps them."""

import pytest
import torch

from serving_ref import DEV, F32, U, Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv", [2, 5, 8, 33, 200])
@pytest.mark.parametrize("n", [1, 2])
def test_weights_over_a_bf16_cache(lib, dim, kv, n):
    """A weight is split into two bf16 parts, the second rounded by 2^-8 of itself: 2^-16 of the
    weight.  The scores' error as in attention64; the result is rounded to bf16 once."""
    p = Paged(lib, [(n, kv)], 8, 2, dim, 16, "bf16", seed=kv, spread=0.5)
    i = torch.arange(kv, device=DEV)
    v = torch.where((i % 2 == 0)[:, None, None], 1.0, -1.0) * (p.rows64(0, "v")[:1] + 0.01 * p.rows64(0, "v"))
    lib.kv_append(p.cache, p.rows64(0, "k").to(torch.bfloat16), v.to(torch.bfloat16),
                  p.table[0].long()[i // 16] * 16 + i % 16)
    out = lib.paged_attention(p.q, p.cache, p.batch).double()
    q, k, v = p.q.double(), *(p.rows64(0, x).repeat_interleave(4, 1) for x in "kv")
    see = i[None, :] <= kv - n + torch.arange(n, device=DEV)[:, None]
    s = torch.einsum("nhd,lhd->hnl", q, k) * dim ** -0.5
    ds = torch.einsum("nhd,lhd->hnl", q.abs(), k.abs()) * dim ** -0.5 * (dim + 4) * F32
    w = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
    ref = torch.einsum("hnl,lhd->nhd", w, v)
    mag = torch.einsum("hnl,lhd->nhd", w, v.abs())
    dmax = torch.where(see, ds, 0.0).amax(-1).T
    bound = U * ref.abs() + (2.0 ** -16 + 2.5 * dmax[..., None] + 2.0 ** -18) * mag
    over = float(((out - ref).abs() / (1.01 * bound)).max())
    assert over <= 1.0, f"{over:.3g} times the bound"


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("kv", [1, 2, 9, 200])
@pytest.mark.parametrize("sign", [1, -1])
def test_an_infinity_that_is_seen_stays_one(lib, dim, kv, sign):
    p = Paged(lib, [(1, kv)], 8, 2, dim, 16, "bf16", seed=kv, spread=0.5)
    p.cache.v[p.table[0, 0], :, 0, ::3] = sign * float("inf")
    out = lib.paged_attention(p.q, p.cache, p.batch)
    assert bool((out[..., ::3] == sign * float("inf")).all())
    assert bool(torch.isfinite(out[..., 1::3]).all())
