"""More of the serving operators' range: batches beyond a block's threads, sequences of many
row tiles, every format under growing, negative and zero score scales, q as a transposed view,
windows with rows that see nothing, idle sequences beside a chunk, 8-bit caches held to the
rounding that f16 weights promise, and the tables' magnitude."""

import math

import pytest
import torch

from serving_ref import DEV, F32, Paged, rope_inputs
from test_serving_scales import check8

pytestmark = pytest.mark.gpu

FMT = pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])


def run(p, lib, **kw):
    lse = torch.empty(p.q.shape[:2], device=DEV)
    out = lib.paged_attention(p.q, p.cache, p.batch, lse=lse, **kw)
    assert lib.poll_status() == 0
    return out, lse


@FMT
@pytest.mark.parametrize("most,hq,hk,dim", [(1, 8, 2, 64), (9, 8, 2, 64), (60, 8, 2, 64), (1, 4, 4, 256), (40, 2, 2, 256)])
def test_more_sequences_than_a_block_has_threads(lib, fmt, most, hq, hk, dim):
    g = torch.Generator().manual_seed(most)
    kv = torch.randint(0, 90, (650,), generator=g).tolist()
    n = torch.randint(0, most + 1, (650,), generator=g).tolist()
    n[-1], kv[-1] = most, 89
    p = Paged(lib, list(zip(n, kv)), hq, hk, dim, 16, fmt, seed=most)
    p.check(*run(p, lib))


@FMT
def test_a_sequence_of_many_row_tiles(lib, fmt):
    p = Paged(lib, [(3, 50), (2300, 2400), (1, 7)], 8, 1, 64, 64, fmt)      # 72 tiles of 32 tokens
    p.check(*run(p, lib))


@FMT
@pytest.mark.parametrize("window", [0, 100])
def test_a_chunk_beside_idle_sequences(lib, fmt, window):
    """The few-row kernel with 75 row tiles in one sequence."""
    p = Paged(lib, [(0, 20)] * 50 + [(300, 500)] + [(0, 0)] * 49, 8, 2, 64, 16, fmt)
    p.check(*run(p, lib, window=window), window=window)


@FMT
@pytest.mark.parametrize("n", [1, 30, 200])
@pytest.mark.parametrize("scale,spread", [(1.0, 4.0), (0.01, 1.0), (-0.3, 2.0), (0.0, 1.0)])
def test_score_scales(lib, fmt, n, scale, spread):
    p = Paged(lib, [(n, 600)], 8, 2, 128, 32, fmt, spread=spread)
    # (8-bit: f16 weights also have a smallest step, which the bf16 bound leaves out)
    check = p.check if fmt == "bf16" else lambda out, lse, scale: check8(p, out, lse, scale=scale)
    check(*run(p, lib, scale=scale), scale=scale)


@FMT
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("n", [1, 30, 200])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_grow_or_fall_along_the_sequence(lib, fmt, dim, n, sign):
    p = Paged(lib, [(n, 1500)], 4, 1, dim, 64, fmt)
    i = torch.arange(1500, device=DEV)
    k = (p.rows64(0, "k") * 0 + 1) * (sign * i / 100.0)[:, None, None]
    p.q.fill_(1.0)
    lib.kv_append(p.cache, k.to(torch.bfloat16), p.rows64(0, "v").to(torch.bfloat16),
                  p.table[0].long()[i // 64] * 64 + i % 64)
    p.check(*run(p, lib))


@FMT
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 30, 150])
def test_q_as_a_transposed_view(lib, fmt, dim, n):
    p = Paged(lib, [(n, 400), (n, 90 + n)], 8, 2, dim, 32, fmt)
    want, _ = run(p, lib)
    flat, p.q = p.q, p.q.transpose(0, 1).contiguous().transpose(0, 1)
    assert p.q.stride() != flat.stride() or n == 0
    got, lse = run(p, lib)
    assert torch.equal(got, want)
    p.check(got, lse)


@FMT
@pytest.mark.parametrize("n,kv", [(5, 2), (40, 30), (200, 30)])
def test_rows_that_a_window_and_the_mask_leave_empty(lib, fmt, n, kv):
    """More new tokens than positions: the first see nothing, with a window too."""
    p = Paged(lib, [(n, kv), (1, 40)], 8, 2, 64, 16, fmt)
    out, lse = run(p, lib, window=8)
    p.check(out, lse, window=8)
    assert bool((out[:n - kv] == 0).all()) and bool(torch.isneginf(lse[:n - kv]).all())


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("lengths,hq,hk,dim", [
    ([(1, 1)], 8, 2, 64), ([(1, 300)], 8, 2, 128), ([(1, 2000)], 16, 16, 256), ([(1, 65), (3, 7), (1, 900)], 14, 2, 64),
    ([(30, 200)], 8, 2, 64), ([(64, 64), (17, 1000)], 16, 2, 128), ([(300, 700), (129, 129)], 8, 2, 128),
    ([(90, 500)], 4, 2, 256),
])
def test_8bit_caches_to_f16_rounding(lib, fmt, lengths, hq, hk, dim):
    p = Paged(lib, lengths, hq, hk, dim, 32, fmt, seed=hq)
    out, lse = run(p, lib)
    for b in range(len(lengths)):
        check8(p, out, lse, b)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_magnitude_of_scaled_tables(lib, layout):
    """It multiplies cos and sin, whatever the scaling; 0 stands for the scaling's own."""
    kinds = [dict(kind="plain"), dict(kind="linear", factor=4.0),
             dict(kind="yarn", factor=16.0, original_len=2048.0), dict(kind="yarn", factor=16.0, original_len=2048.0)]
    own = [1.0, 1.0, 0.1 * math.log(16.0) + 1.0, 0.1 * math.log(16.0) + 1.0]
    for kw, m0, m in zip(kinds, own, (0.5, 1.7, 1.0, 3.0)):
        base = lib.rope_table_scaled(300, 64, 10000.0, dict(kw), device=DEV)
        got = lib.rope_table_scaled(300, 64, 10000.0, dict(kw, magnitude=m), device=DEV)
        for a, b in zip(got, base):
            # one rounding to f32 on either side
            assert float((a.double() - b.double() * (m / m0)).abs().max()) <= 2 * F32 * m * 1.001
    # and the rotation takes them as they are
    q = torch.ones(300, 1, 64, dtype=torch.bfloat16, device=DEV)
    rope = rope_inputs(300, 64, layout)
    y1 = lib.rotary(q, rope=rope)
    y2 = lib.rotary(q, rope={**rope, "cos": rope["cos"] * 2, "sin": rope["sin"] * 2})
    assert torch.equal(y2, y1 * 2)
