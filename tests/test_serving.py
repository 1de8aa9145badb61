"""Rotary positions, the paged cache and the attention over it against plain 64-bit forms
(serving_ref.py), at the sizes and masks where they can go wrong: one token to long ones,
odd lengths, pages that end inside a tile, strided views, every format, rows whose mask
leaves nothing, garbage past a sequence's end."""

import math

import pytest
import torch

from serving_ref import (DEV, F32, TOP, U, Paged, cache_values64, check_rotated, rope_inputs, rotate64, tables64)

pytestmark = pytest.mark.gpu


def _bf16(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _packed(tokens, hq, hk, dim, seed=0):
    """q, k, v as slices of one [tokens, (hq + 2 hk) dim] buffer."""
    buf = _bf16(tokens, (hq + 2 * hk) * dim, seed=seed)
    q, k, v = buf.split([hq * dim, hk * dim, hk * dim], 1)
    return tuple(t.unflatten(1, (h, dim)) for t, h in ((q, hq), (k, hk), (v, hk)))


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [
    (1, 1, 1, 64, 64), (7, 14, 2, 64, 32), (33, 3, 1, 128, 128), (130, 16, 16, 256, 64), (5, 2, 1, 96, 48),
    (9, 4, 2, 64, 2), (11, 4, 2, 128, 20), (3, 2, 1, 8, 6), (2000, 32, 8, 128, 128), (4, 1, 1, 1024, 1024),
])
def test_rotary(lib, tokens, hq, hk, dim, rot, layout):
    q, k, _ = _packed(tokens, hq, hk, dim, seed=tokens)
    rope = rope_inputs(tokens, rot, layout, seed=rot)
    for inverse in (False, True):
        yq, yk = lib.rotary(q, k, rope=rope, inverse=inverse)
        check_rotated(yq, q, rope, inverse)
        check_rotated(yk, k, rope, inverse)
        assert torch.equal(yq[..., rot:], q[..., rot:])
        only = lib.rotary(q, rope=rope, inverse=inverse)
        assert torch.equal(only, yq)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 64), ("half", 20), ("interleaved", 128),
                                        ("interleaved", 22)])
def test_rotary_in_place_and_strided_outputs(lib, layout, rot):
    q, k, _ = _packed(300, 8, 2, 128, seed=3)
    rope = rope_inputs(300, rot, layout)
    yq, yk = lib.rotary(q, k, rope=rope)
    heads_first = torch.empty(8, 300, 128, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    lib.rotary(q, k, rope=rope, q_out=heads_first, k_out=k)
    assert torch.equal(heads_first, yq) and torch.equal(k, yk)
    lib.rotary(q, rope=rope, q_out=q)
    assert torch.equal(q, yq)


def test_rotary_position_outside_the_table_is_reported(lib):
    q = _bf16(6, 2, 64)
    rope = rope_inputs(6, 64, "half")
    rope["pos"][2], rope["pos"][4] = -1, 500
    y = lib.rotary(q, rope=rope)
    assert lib.poll_status() == 7
    rope["pos"][2], rope["pos"][4] = 0, 0
    assert torch.equal(lib.rotary(q, rope=rope), y)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_gradient(lib, layout):
    """autograd against the transpose rotation and against central differences of the
    64-bit form along random directions (the map is linear: the difference is exact up to
    the rounding of the kernel's own gradient)."""
    from rank_mlp_gb300.autograd import lora_rotary
    q, k, _ = (t.contiguous().requires_grad_() for t in _packed(17, 4, 2, 64, seed=5))
    rope = rope_inputs(17, 48, layout)
    yq, yk = lora_rotary(q, k, rope)
    gq, gk = _bf16(17, 4, 64, seed=6), _bf16(17, 2, 64, seed=7)
    torch.autograd.backward([yq, yk], [gq, gk])
    check_rotated(q.grad, gq, rope, inverse=True)
    check_rotated(k.grad, gk, rope, inverse=True)
    for x, dy, dx in ((q, gq, q.grad), (k, gk, k.grad)):
        v = torch.randn(x.shape, dtype=torch.float64, device=DEV, generator=torch.Generator(DEV).manual_seed(8))
        f = lambda t: float((rotate64(t, rope)[0] * dy.double()).sum())  # noqa: E731
        diff = (f(x.detach().double() + v) - f(x.detach().double() - v)) / 2
        got = float((dx.double() * v).sum())
        assert abs(got - diff) <= 2 * U * float((dx.double().abs() * v.abs()).sum())


def _scaled64(n_pos, rot, base, kind, factor=1.0, length=0.0, low=1.0, high=32.0):
    """Frequencies from the definitions in the header, column by column."""
    w, mag = [], 1.0
    for c in range(rot // 2):
        f = base ** (-2.0 * c / rot)
        if kind == "linear":
            f /= factor
        elif kind == "ntk":
            f = (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * c / rot)
        elif kind == "yarn":
            at = lambda turns: rot * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
            g = min(max((c - lo) / (hi - lo), 0.0), 1.0)
            f, mag = (1 - g) * f + g * f / factor, 0.1 * math.log(factor) + 1
        elif kind == "wavelength":
            lam = 2 * math.pi / f
            if lam > length / low:
                f /= factor
            elif lam >= length / high:
                g = (length / lam - low) / (high - low)
                f = g * f + (1 - g) * f / factor
        w.append(f)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * torch.tensor(w, dtype=torch.float64)
    return mag * a.cos(), mag * a.sin()


@pytest.mark.parametrize("rot,kw", [
    (64, dict(kind="plain")), (128, dict(kind="linear", factor=4.0)), (128, dict(kind="ntk", factor=8.0)),
    (64, dict(kind="yarn", factor=16.0, original_len=2048.0, low=1.0, high=32.0)),
    (128, dict(kind="wavelength", factor=8.0, original_len=4096.0, low=1.0, high=4.0)),
    (6, dict(kind="ntk", factor=2.0)),
])
def test_scaled_tables(lib, rot, kw):
    cos, sin = lib.rope_table_scaled(6000, rot, 500000.0, dict(kw), device=DEV)
    args = dict(kw)
    if "original_len" in args:
        args["length"] = args.pop("original_len")
    rc, rs = _scaled64(6000, rot, 500000.0, **args)
    # one rounding to f32 of values up to the magnitude (1.28 at most), and the 64-bit
    # angle (up to 6000) times the frequency's few ulps
    assert float((cos.cpu().double() - rc).abs().max()) <= 1.3 * F32 + 6000 * 2.0 ** -48
    assert float((sin.cpu().double() - rs).abs().max()) <= 1.3 * F32 + 6000 * 2.0 ** -48
    if kw["kind"] == "plain":
        pc, ps = lib.rope_table(6000, rot, 500000.0, device=DEV)
        assert torch.equal(pc, cos) and torch.equal(ps, sin)


# ------------------------------------------------------------------ the cache

def _quant32(y, fmt):
    """Codes and scales by the definition, in f32 (every operation rounded)."""
    amax = y.abs().amax(-1, keepdim=True)
    scale = (amax * (1.0 / TOP[fmt])).clamp_min(1.17549435e-38)
    fine = torch.isfinite(amax)
    z = torch.where(fine, y * torch.reciprocal(scale), torch.zeros_like(y)).clamp(-TOP[fmt], TOP[fmt])
    scale = torch.where(fine, scale, torch.full_like(scale, math.nan))
    code = z.round().to(torch.int8) if fmt == "int8" else z.to(torch.float8_e4m3fn)
    return code, scale.squeeze(-1)


def _turn32(x, rope):
    x = x.float()
    h = rope["cos"].shape[1]
    c, s = (rope[n][rope["pos"].long()][:, None] for n in ("cos", "sin"))
    ia = torch.arange(h, device=DEV) * (1 if rope["layout"] == "half" else 2)
    ib = ia + (h if rope["layout"] == "half" else 1)
    y = x.clone()
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    return y


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,layout,page", [
    (1, 4, 1, 64, 64, "half", 16), (37, 14, 2, 64, 32, "interleaved", 32), (65, 8, 8, 128, 128, "half", 16),
    (19, 4, 2, 256, 256, "half", 128), (6, 6, 3, 128, 20, "half", 64), (6, 6, 3, 128, 22, "interleaved", 256),
    (3001, 4, 2, 128, 128, "interleaved", 64), (8, 0, 2, 64, 0, "half", 16),
])
def test_append_rotates_quantises_and_scatters(lib, tokens, hq, hk, dim, rot, layout, page, fmt):
    q, k, v = _packed(tokens, max(hq, 1), hk, dim, seed=tokens + dim)
    rope = rope_inputs(tokens, rot, layout, seed=1) if rot else None
    cache = lib.kv_cache(2 * (-(-tokens // page)) + 1, page, hk, dim, fmt, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    slots = torch.randperm(cache.n_pages * page, generator=g, device=DEV)[:tokens]
    slots[tokens // 2] = -5 if tokens > 1 else slots[0]        # padding
    live = slots >= 0
    yq = lib.kv_append(cache, k, v, slots, q=q if hq else None, rope=rope)
    if hq:
        check_rotated(yq, q, rope)
    else:
        assert yq is None
    at, off = slots[live] // page, slots[live] % page
    written = torch.zeros(cache.n_pages, page, dtype=torch.bool, device=DEV)
    written[at, off] = True
    for n, x in (("k", _turn32(k, rope) if rot else k.float()), ("v", v.float())):
        got = getattr(cache, n)
        raw = got.view(torch.uint8) if fmt != "bf16" else got
        assert not bool(raw.transpose(1, 2)[~written].any()), "a slot that is not in the call was written"
        if fmt == "bf16":
            assert torch.equal(got[at, :, off], x[live].to(torch.bfloat16))
            continue
        code, scale = _quant32(x[live], fmt)
        sc = getattr(cache, n + "_scale")
        assert torch.equal(sc[at, :, off], scale)
        assert torch.equal(raw[at, :, off], code.view(torch.uint8))
        # what the codes stand for, against the 64-bit rotation: half a step of the format
        ref = (rotate64(k, rope)[0] if n == "k" and rot else x.double())[live]
        val = cache_values64(cache, n)[at, :, off]
        s = scale.double()[..., None]
        step = 0.5 * s if fmt == "int8" else torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * s)
        assert bool(((val - ref).abs() <= step * 1.001 + 8 * F32 * ref.abs().amax(-1, keepdim=True)).all())
    assert lib.poll_status() == 0


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
def test_append_of_zero_tiny_huge_and_broken_rows(lib, fmt):
    k = torch.zeros(8, 1, 64, dtype=torch.bfloat16, device=DEV)
    k[1] = 1e-40
    k[2] = 3e38
    k[3, 0, 5] = math.inf
    k[4, 0, 7] = math.nan
    k[5, 0, 0] = -0.0
    k[6, 0, ::2] = -1.0
    v = _bf16(8, 1, 64)
    cache = lib.kv_cache(1, 16, 1, 64, fmt, device=DEV)
    lib.kv_append(cache, k, v, torch.arange(8, device=DEV))
    code, scale = _quant32(k.float(), fmt)
    assert torch.equal(cache.k_scale[0, 0, :8].isnan(), scale[:, 0].isnan())
    assert torch.equal(cache.k_scale[0, 0, :8].nan_to_num(), scale[:, 0].nan_to_num())
    assert torch.equal(cache.k.view(torch.uint8)[0, 0, :8], code.view(torch.uint8)[:, 0])
    assert bool(cache.k_scale[0, 0, 3:5].isnan().all())
    kk, _ = lib.kv_read(cache, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                        torch.tensor([0, 8], dtype=torch.int32, device=DEV), 8)
    assert bool(kk[3:5].isnan().all()) and bool(torch.isfinite(kk[[0, 1, 2, 5, 6, 7]]).all())
    assert bool((kk[0] == 0).all())


def test_append_slot_past_the_cache_is_skipped_and_reported(lib):
    cache = lib.kv_cache(2, 16, 2, 64, "int8", device=DEV)
    k, v = _bf16(3, 2, 64), _bf16(3, 2, 64, seed=1)
    lib.kv_append(cache, k, v, torch.tensor([31, 32, 1 << 40], device=DEV))
    assert lib.poll_status() == 7
    assert bool(cache.k[1, :, 15].any()) and not bool(cache.k[0].any()) and not bool(cache.k[1, :, :15].any())
    assert lib.poll_status() == 0


def test_append_q_in_place(lib):
    q, k, v = _packed(50, 6, 2, 128, seed=9)
    for rot, layout in ((128, "half"), (20, "half"), (64, "interleaved")):
        rope = rope_inputs(50, rot, layout)
        cache = lib.kv_cache(4, 16, 2, 128, "bf16", device=DEV)
        y = lib.kv_append(cache, k, v, torch.arange(50, device=DEV), q=q, rope=rope)
        q2 = q.clone()
        lib.kv_append(cache, k, v, torch.arange(50, device=DEV), q=q2, rope=rope, q_out=q2)
        assert torch.equal(q2, y)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("lengths,hk,dim,page", [
    ([1], 1, 64, 16), ([0, 17, 0, 0, 33, 1], 3, 128, 16), ([300, 5, 129], 2, 256, 128), ([2000, 1], 8, 128, 64),
])
def test_read_back(lib, lengths, hk, dim, page, fmt):
    p = Paged(lib, [(0, n) for n in lengths], hk, hk, dim, page, fmt, seed=len(lengths))
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=DEV)
    k, v = lib.kv_read(p.cache, p.table, cu, sum(lengths))
    for got, n in ((k, "k"), (v, "v")):
        ref = torch.cat([p.rows64(b, n) for b in range(len(lengths))])
        # code times scale rounded to f32, then to bf16
        assert bool(((got.double() - ref).abs() <= (U + 2 * F32) * ref.abs()).all())
    assert lib.poll_status() == 0


def test_read_reports_what_it_cannot_read(lib):
    p = Paged(lib, [(0, 20)], 2, 2, 64, 16, "int8")
    for cu, total, zero in (([0, 20], 24, slice(20, 24)), ([2, 20], 20, slice(0, 2)), ([0, 40], 40, slice(32, 40))):
        k, _ = lib.kv_read(p.cache, p.table, torch.tensor(cu, dtype=torch.int32, device=DEV), total)
        assert lib.poll_status() == 7
        assert bool((k[zero] == 0).all())
    bad = p.table.clone()
    bad[0, 1] = p.cache.n_pages
    k, _ = lib.kv_read(p.cache, bad, torch.tensor([0, 20], dtype=torch.int32, device=DEV), 20)
    assert lib.poll_status() == 7 and bool((k[16:] == 0).all())


# ------------------------------------------------------------------ attention

FORMATS = ["bf16", "fp8", "int8"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths,hq,hk,dim,page", [
    ([(1, 1)], 1, 1, 64, 16),
    ([(1, 777)], 14, 2, 64, 16),
    ([(1, 5), (1, 64), (1, 65), (1, 1), (1, 1000), (1, 128)], 32, 8, 128, 64),
    ([(1, 300)] * 3, 16, 16, 256, 32),
    ([(1, 4100), (1, 17)], 8, 1, 128, 256),
    ([(1, 333), (1, 2)], 40, 1, 64, 16),                      # more heads share one than a tile has rows
])
def test_decode(lib, lengths, hq, hk, dim, page, fmt):
    p = Paged(lib, lengths, hq, hk, dim, page, fmt, seed=dim + hq)
    lse = torch.empty(p.q.shape[:2], device=DEV)
    out = lib.paged_attention(p.q, p.cache, p.batch, lse=lse)
    p.check(out, lse)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths,hq,hk,dim,page", [
    ([(2, 2)], 4, 4, 64, 16),
    ([(129, 129)], 4, 2, 64, 16),                             # a first prefill, odd
    ([(127, 500), (64, 64), (3, 700)], 14, 2, 64, 32),        # seven heads share one
    ([(300, 300), (1, 300), (0, 40), (256, 1029)], 8, 2, 128, 64),
    ([(640, 640)], 4, 4, 128, 128),
    ([(200, 200), (77, 390)], 4, 2, 256, 32),
    ([(33, 2000)], 2, 2, 256, 16),
    ([(17, 3000)], 16, 1, 128, 64),
])
def test_chunks(lib, lengths, hq, hk, dim, page, fmt):
    p = Paged(lib, lengths, hq, hk, dim, page, fmt, seed=dim + hq, strided=True)
    lse = torch.empty(p.q.shape[:2], device=DEV)
    out = lib.paged_attention(p.q, p.cache, p.batch, lse=lse)
    p.check(out, lse)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 50), (True, 128), (False, 0), (False, 60)])
def test_masks(lib, causal, window, dim, fmt):
    p = Paged(lib, [(200, 300), (1, 257), (5, 5), (140, 140)], 8, 2, dim, 32, fmt, seed=window)
    lse = torch.empty(p.q.shape[:2], device=DEV)
    out = lib.paged_attention(p.q, p.cache, p.batch, causal=causal, window=window, lse=lse)
    p.check(out, lse, causal=causal, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lengths", [
    [(3, 0), (1, 0), (1, 40)],            # nothing cached
    [(9, 4), (1, 20), (200, 150)],        # more new tokens than positions: the first see nothing
])
def test_tokens_that_see_nothing(lib, lengths, dim, fmt):
    p = Paged(lib, lengths, 8, 4, dim, 16, fmt)
    lse = torch.empty(p.q.shape[:2], device=DEV)
    out = torch.full(p.q.shape, math.nan, dtype=torch.bfloat16, device=DEV)
    lib.paged_attention(p.q, p.cache, p.batch, lse=lse, out=out)
    p.check(out, lse)
    b, (n, kv) = next((i, l) for i, l in enumerate(lengths) if l[0] > l[1])
    blind = slice(p.cu[b], p.cu[b] + n - kv)
    assert bool((out[blind] == 0).all()) and bool(torch.isneginf(lse[blind]).all())
    assert lib.poll_status() == 0


@pytest.mark.parametrize("rows", [1, 150])
def test_window_that_leaves_a_row_empty(lib, rows):
    """Without the causal mask a token before position 0 (more new tokens than positions)
    has window positions only past the sequence's start."""
    p = Paged(lib, [(rows + 30, 30)], 4, 2, 64, 16, "bf16")
    out = lib.paged_attention(p.q, p.cache, p.batch, causal=False, window=8)
    p.check(out, causal=False, window=8)


@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("scale,spread", [(1.0, 4.0), (0.01, 1.0), (-0.3, 2.0), (0.0, 1.0)])
def test_score_scales(lib, n, scale, spread):
    """Weights from all equal to a single one (scores up to hundreds)."""
    p = Paged(lib, [(n, 600)], 8, 2, 128, 32, "bf16", spread=spread)
    out = lib.paged_attention(p.q, p.cache, p.batch, scale=scale)
    p.check(out, scale=scale)


@pytest.mark.parametrize("n", [1, 160])
def test_growing_scores(lib, n):
    """Keys that grow along the sequence: the running maximum rises at every tile."""
    p = Paged(lib, [(n, 1500)], 4, 1, 64, 64, "bf16")
    i = torch.arange(1500, device=DEV)
    k = (p.rows64(0, "k") * 0 + 1) * (i / 100.0)[:, None, None]
    p.q.fill_(1.0)
    lib.kv_append(p.cache, k.to(torch.bfloat16), p.rows64(0, "v").to(torch.bfloat16),
                  p.table[0].long()[i // 64] * 64 + i % 64)
    out = lib.paged_attention(p.q, p.cache, p.batch)
    p.check(out)


def test_ragged_batch_of_everything(lib):
    g = torch.Generator().manual_seed(4)
    for n in (1, 3, 40):
        kv = torch.randint(1, 1500, (n,), generator=g).tolist()
        new = [min(k, int(x)) for k, x in zip(kv, torch.randint(0, 90, (n,), generator=g))]
        p = Paged(lib, list(zip(new, kv)), 12, 4, 64, 16, "fp8", seed=n, strided=True)
        out = lib.paged_attention(p.q, p.cache, p.batch)
        p.check(out)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hk,dim,new", [(16, 8, 64, (1, 90)), (16, 8, 128, (1, 90)), (32, 4, 64, (1, 90)),
                                           (32, 4, 128, (1, 90)), (8, 8, 256, (1, 200)), (16, 2, 256, (1, 40)),
                                           (16, 8, 128, (1, 3)), (8, 8, 256, (1, 3))])
def test_many_items_for_each_block(lib, hq, hk, dim, new, fmt):
    """More (sequence, head, row tile) items than the GPU has blocks, in every kernel: blocks go
    from one item to the next, with one and with two row halves, whole items and cut ones."""
    g = torch.Generator().manual_seed(dim + hq)
    kv = torch.randint(1, 700, (120,), generator=g).tolist()
    n = torch.randint(new[0], new[1] + 1, (120,), generator=g).tolist()
    p = Paged(lib, [(min(a, b), b) for a, b in zip(n, kv)], hq, hk, dim, 32, fmt, seed=hq)
    lse = torch.empty(p.q.shape[:2], device=DEV)
    out = lib.paged_attention(p.q, p.cache, p.batch, lse=lse)
    assert lib.poll_status() == 0
    p.check(out, lse)


def test_repeated_calls_and_graph_replays_give_the_same_bits(lib):
    p = Paged(lib, [(1, 3000), (1, 7), (90, 1000)], 8, 2, 128, 64, "int8")
    first = lib.paged_attention(p.q, p.cache, p.batch)
    for _ in range(3):
        assert torch.equal(lib.paged_attention(p.q, p.cache, p.batch), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.paged_attention(p.q, p.cache, p.batch)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = lib.paged_attention(p.q, p.cache, p.batch)
    for kv in (3000, 1234, 2999):          # lengths change on the device between replays
        p.kv_len[0] = kv
        p.lengths[0] = (1, kv)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        p.check(out)
    assert lib.poll_status() == 0


def test_other_stream(lib):
    p = Paged(lib, [(1, 900), (60, 200)], 8, 2, 64, 16, "bf16")
    torch.cuda.synchronize()
    ref = lib.paged_attention(p.q, p.cache, p.batch)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out = lib.paged_attention(p.q, p.cache, p.batch)
    s.synchronize()
    assert torch.equal(out, ref)


def test_values_on_the_device_that_are_out_of_range(lib):
    """A page outside the cache, a length past the table, query rows outside q: reported,
    cut to what there is, and other sequences are untouched."""
    p = Paged(lib, [(1, 100), (2, 60)], 4, 2, 64, 16, "int8")
    good = lib.paged_attention(p.q, p.cache, p.batch)
    table = p.table.clone()
    table[0, 3] = 1 << 30
    out = lib.paged_attention(p.q, p.cache, lib.paged_batch(table, p.kv_len, p.cu_q))
    assert lib.poll_status() == 7
    assert torch.equal(out[1:], good[1:])
    table[0, 3] = -1
    lib.paged_attention(p.q, p.cache, lib.paged_batch(table, p.kv_len, p.cu_q))
    assert lib.poll_status() == 7
    for kv in (10 ** 9, -3):
        long = p.kv_len.clone()
        long[0] = kv
        out = lib.paged_attention(p.q, p.cache, lib.paged_batch(p.table, long, p.cu_q))
        assert lib.poll_status() == 7
        assert torch.equal(out[1:], good[1:])
    for cu in ([0, 1, 1 << 30], [-4, 1, 3], [0, 2, 1]):
        lib.paged_attention(p.q, p.cache, lib.paged_batch(p.table, p.kv_len,
                                                          torch.tensor(cu, dtype=torch.int32, device=DEV)))
        assert lib.poll_status() == 7
    out = torch.full(p.q.shape, 3.0, dtype=torch.bfloat16, device=DEV)      # rows nobody owns stay
    lib.paged_attention(p.q, p.cache, lib.paged_batch(p.table, p.kv_len,
                                                      torch.tensor([1, 1, 3], dtype=torch.int32, device=DEV)), out=out)
    assert lib.poll_status() == 0
    assert bool((out[0] == 3.0).all()) and torch.equal(out[1:], good[1:])


def test_no_tokens(lib):
    cache = lib.kv_cache(2, 16, 2, 64, "fp8", device=DEV)
    e = lambda h: torch.empty(0, h, 64, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    n0 = lib.launch_count()
    rope = rope_inputs(0, 64, "half")
    assert lib.rotary(e(4), e(2), rope=rope)[0].shape == (0, 4, 64)
    assert lib.kv_append(cache, e(2), e(2), torch.empty(0, dtype=torch.int64, device=DEV), q=e(4), rope=rope).numel() == 0
    b = lib.paged_batch(torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV),
                        torch.zeros(2, dtype=torch.int32, device=DEV))
    assert lib.paged_attention(e(4), cache, b).shape == (0, 4, 64)
    assert lib.kv_read(cache, b.page_table, b.cu_q, 0)[0].numel() == 0
    assert lib.launch_count() == n0


@pytest.mark.slow
def test_a_cache_past_32_bit_offsets(lib):
    """Pages whose element offsets pass 2^32: the last pages of a 10 GB pool."""
    D, hk, page = 256, 16, 256
    n_pages = (1 << 32) // (D * hk * page) + 4
    cache = lib.kv_cache(n_pages, page, hk, D, "bf16", device=DEV)
    k, v = _bf16(300, hk, D), _bf16(300, hk, D, seed=1)
    i = torch.arange(300, device=DEV)
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device=DEV)
    lib.kv_append(cache, k, v, table[0].long()[i // page] * page + i % page)
    kk, vv = lib.kv_read(cache, table, torch.tensor([0, 300], dtype=torch.int32, device=DEV), 300)
    assert torch.equal(kk, k) and torch.equal(vv, v)
    from serving_ref import attention64
    for n in (1, 200):
        q = _bf16(n, hk, D, seed=2)
        b = lib.paged_batch(table, torch.tensor([300], dtype=torch.int32, device=DEV),
                            torch.tensor([0, n], dtype=torch.int32, device=DEV))
        out = lib.paged_attention(q, cache, b)
        ref, _, bound, _ = attention64(q, k, v, 300 - n, D ** -0.5)
        assert bool(((out.double() - ref).abs() <= 1.01 * bound).all())
