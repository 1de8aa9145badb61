"""Attention over 8-bit caches whose rows of V differ in size by many powers of two: per row,
per tile, in a position that carries no weight and in one that the mask hides.  Both kernels
(few and many query rows) are held to what f16 weights promise, 2^-11 each, so an answer
does not depend on which of them a batch's size picks."""

import math

import pytest
import torch

from serving_ref import DEV, F32, TOP, U, Paged

pytestmark = pytest.mark.gpu

F16 = 2.0 ** -11


def fill(p, lib, b, k=None, v=None):
    """Writes sequence b's K and V anew ([kv, hk, D], any float type)."""
    kv, page = p.lengths[b][1], p.cache.page_size
    i = torch.arange(kv, device=DEV)
    slots = p.table[b].long()[i // page] * page + i % page
    rows = [(p.rows64(b, n) if x is None else x).to(torch.bfloat16) for n, x in (("k", k), ("v", v))]
    lib.kv_append(p.cache, *rows, slots)


def scales64(p, b):
    """V's scales of sequence b, [kv, hk] in 64 bits."""
    t = p.cache.v_scale[p.table[b].long()].double()
    return t.transpose(1, 2).flatten(0, 1)[:p.lengths[b][1]]


def check8(p, out, lse, b=0, causal=True, window=0, scale=None):
    """Sequence b against the definition in 64 bits.

    Weights are rounded to f16: by 2^-11 of each or, where they are small, by 2^-25 of the
    largest weight times scale (times the largest code).  The many-row kernel also rounds V to
    2^-11 of itself or, for the smallest e4m3 codes, 2^-26 of the row's largest.  Scores as in
    attention64; the result is rounded to bf16 once."""
    n, kv = p.lengths[b]
    fmt = "int8" if p.cache.k.dtype == torch.int8 else "fp8"
    g = p.hq // p.hk
    q = p.q[p.cu[b]:p.cu[b] + n].double()
    k, v, sc = (x.repeat_interleave(g, 1) for x in (p.rows64(b, "k"), p.rows64(b, "v"), scales64(p, b)))
    pos = kv - n + torch.arange(n, device=DEV)[:, None]
    j = torch.arange(kv, device=DEV)[None, :]
    see = j <= pos if causal else j > -1 - 0 * pos
    if window:
        see = see & (pos - j < window)
    scale = p.D ** -0.5 if scale is None else scale
    s = torch.einsum("nhd,lhd->hnl", q, k) * scale
    ds = torch.einsum("nhd,lhd->hnl", q.abs(), k.abs()) * abs(scale) * (p.D + 4) * F32
    s = s.masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - top)
    tot = w.sum(-1, keepdim=True)
    w = w / tot
    v = torch.where(torch.isnan(v), 0.0, v)              # hidden ones only: see the callers
    sc = torch.where(torch.isnan(sc), 0.0, sc)
    ref = torch.einsum("hnl,lhd->nhd", w, v)
    mag = torch.einsum("hnl,lhd->nhd", w, v.abs())
    each = w * (sc * TOP[fmt]).T[:, None, :]             # weight times the largest value of a row
    dmax = torch.where(see, ds, 0.0).amax(-1).T
    small = (see.sum(-1)[None, :] * 2.0 ** -25 * each.amax(-1) + 2.0 ** -26 * each.sum(-1)).T
    bound = U * ref.abs() + (2 * F16 + 2.5 * dmax[..., None] + 2.0 ** -17) * mag + small[..., None]
    got = out[p.cu[b]:p.cu[b] + n].double()
    assert bool(torch.isfinite(got).all())
    over = float(((got - ref).abs() / (1.01 * bound).clamp_min(1e-300)).max())
    assert over <= 1.0, f"{over:.3g} times the bound"
    rl = (top + torch.log(tot)).squeeze(-1).T
    assert bool(((lse[p.cu[b]:p.cu[b] + n].double() - rl).abs() <= dmax + 2.0 ** -17 + rl.abs() * 2.0 ** -20).all())


def run(p, lib, **kw):
    lse = torch.empty(p.q.shape[:2], device=DEV)
    out = lib.paged_attention(p.q, p.cache, p.batch, lse=lse, **kw)
    assert lib.poll_status() == 0
    return out, lse


FMT = pytest.mark.parametrize("fmt", ["fp8", "int8"])
DIM = pytest.mark.parametrize("dim", [64, 128, 256])
NEW = pytest.mark.parametrize("n", [1, 30, 150])      # few rows; one row half; two (one at heads of 256)
KV = 700


def _paged(lib, fmt, dim, n, kv=KV, seed=0, spread=2.0):
    p = Paged(lib, [(n, kv)], 8, 2, dim, 32, fmt, seed=seed + dim + n, spread=spread)
    return p, torch.Generator(device=DEV).manual_seed(seed + 7)


def _rows(p, g):
    return torch.randn(p.lengths[0][1], p.hk, p.D, generator=g, device=DEV, dtype=torch.float64)


@FMT
@DIM
@NEW
@pytest.mark.parametrize("most", [0, 8, 24])
def test_rows_of_v_of_different_size(lib, fmt, dim, n, most):
    p, g = _paged(lib, fmt, dim, n)
    e = torch.randint(0, most + 1, (KV, 2, 1), generator=g, device=DEV)
    fill(p, lib, 0, v=_rows(p, g) * 2.0 ** -e.double())
    check8(p, *run(p, lib))


@FMT
@DIM
@NEW
@pytest.mark.parametrize("step", [-9, -3, 3, 9])
def test_tiles_of_v_of_different_size(lib, fmt, dim, n, step):
    """Sizes that fall or grow from tile to tile, up to 2^100 apart."""
    p, g = _paged(lib, fmt, dim, n)
    e = (torch.arange(KV, device=DEV) // 64 * step).double()[:, None, None]
    fill(p, lib, 0, v=_rows(p, g) * 2.0 ** e)
    check8(p, *run(p, lib))


@FMT
@DIM
@NEW
@pytest.mark.parametrize("more", [8, 16, 20, 26, 60])
@pytest.mark.parametrize("where", ["first tile", "last tile", "one position"])
def test_large_v_without_weight(lib, fmt, dim, n, more, where):
    """Positions with a weight of 2^-60 - more hold a V 2^more times the others'."""
    p, g = _paged(lib, fmt, dim, n)
    p.q.fill_(1.0)
    k, v = _rows(p, g) * 0.05, _rows(p, g)
    at = {"first tile": slice(0, 128), "last tile": slice(384, 512), "one position": slice(300, 301)}[where]
    k[at] = -(60 + more) * math.log(2.0) / math.sqrt(dim)
    v[at] *= 2.0 ** more
    fill(p, lib, 0, k, v)
    check8(p, *run(p, lib))


@FMT
@DIM
@pytest.mark.parametrize("n", [1, 30, 80])
@pytest.mark.parametrize("more", [16, 26, 60])
@pytest.mark.parametrize("where", ["first tile", "last tile"])
def test_large_v_without_weight_in_whole_items(lib, fmt, dim, n, more, where):
    """The same among so many sequences that a block walks whole ones, tile by tile."""
    p = Paged(lib, [(n, 600)] * 160, 8, 2, dim, 32, fmt, seed=dim + n)
    g = torch.Generator(device=DEV).manual_seed(7)
    p.q.fill_(1.0)
    at = slice(0, 128) if where == "first tile" else slice(384, 512)
    for b in (0, 71, 159):
        k, v = _rows(p, g) * 0.05, _rows(p, g)
        k[at] = -(60 + more) * math.log(2.0) / math.sqrt(dim)
        v[at] *= 2.0 ** more
        fill(p, lib, b, k, v)
    out, lse = run(p, lib)
    for b in (0, 71, 159):
        check8(p, out, lse, b)


@FMT
@DIM
@pytest.mark.parametrize("n", [1, 30, 80])
@pytest.mark.parametrize("step", [-13, -6, 6, 13])
def test_tiles_of_different_size_in_whole_items(lib, fmt, dim, n, step):
    """Sizes up to 2^104 apart among tiles that one block walks."""
    p = Paged(lib, [(n, 600)] * 160, 8, 2, dim, 32, fmt, seed=dim + n)
    g = torch.Generator(device=DEV).manual_seed(8)
    for b in (3, 158):
        e = ((torch.arange(600, device=DEV) // 64 - 4) * step).double()[:, None, None]
        fill(p, lib, b, v=_rows(p, g) * 2.0 ** e)
    out, lse = run(p, lib)
    for b in (3, 158):
        check8(p, out, lse, b)


@FMT
@DIM
@NEW
@pytest.mark.parametrize("what", ["2^26", "nan"])
def test_large_and_broken_hidden_v(lib, fmt, dim, n, what):
    """The last position's V, which only the last token sees, and one before every window."""
    p, g = _paged(lib, fmt, dim, n, kv=KV)
    v = _rows(p, g)
    bad = math.nan if what == "nan" else 2.0 ** 26
    v[KV - 1] *= bad
    v[KV - n - 40] *= bad
    fill(p, lib, 0, v=v)
    out, lse = run(p, lib, window=40)
    if what == "nan":
        assert bool(out[n - 1].isnan().all())            # it sees it
        p.lengths[0] = (n - 1, KV - 1)
        p.cu = [0, n - 1]
    if n > 1 or what != "nan":
        check8(p, out, lse, window=40)


@FMT
@NEW
@pytest.mark.parametrize("size", [2.0 ** -115, 2.0 ** -90, 2.0 ** 100, 2.0 ** 112])
def test_v_at_the_ends_of_the_range(lib, fmt, n, size):
    p, g = _paged(lib, fmt, 128, n)
    v = _rows(p, g).clamp(-4, 4)
    fill(p, lib, 0, v=v * size)
    check8(p, *run(p, lib))


@FMT
@NEW
def test_zero_rows_of_v_among_others(lib, fmt, n):
    """A zero row has the smallest scale there is."""
    p, g = _paged(lib, fmt, 128, n)
    v = _rows(p, g)
    v[::3] = 0.0
    v[256:384] = 0.0
    fill(p, lib, 0, v=v)
    check8(p, *run(p, lib))


@FMT
@NEW
def test_joined_parts_of_v_of_different_size(lib, fmt, n):
    """A long sequence, shared out over many blocks whose parts are joined."""
    p, g = _paged(lib, fmt, 128, n, kv=20000)
    e = (torch.arange(20000, device=DEV) // 1000).double()[:, None, None]
    fill(p, lib, 0, v=_rows(p, g) * 2.0 ** (-1.5 * e).floor())
    check8(p, *run(p, lib))
