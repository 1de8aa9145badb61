"""A sliding window over a cache whose old pages have been released: table entries of pages
that lie wholly before what a sequence's first new token sees may hold anything."""

import math

import pytest
import torch

from serving_ref import DEV, Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 30, 150])              # few rows; one row half; two (one at heads of 256)
@pytest.mark.parametrize("page,window,causal", [(16, 40, True), (16, 1, True), (32, 100, False), (128, 130, True)])
def test_released_pages_are_not_looked_at(lib, fmt, dim, n, page, window, causal):
    lengths = [(n, 900), (1, 777), (n, n + 5)]

    def released(p):
        return [(b, max(0, kv - m - window + 1) // page) for b, (m, kv) in enumerate(p.lengths)]

    # page 0, which an entry outside the cache is read as, belongs to nobody's window
    for seed in range(100):
        p = Paged(lib, lengths, 8, 2, dim, page, fmt, seed=seed)
        live = torch.cat([p.table[b, gone:-(-lengths[b][1] // page)] for b, gone in released(p)])
        if not bool((live == 0).any()):
            break
    else:
        pytest.fail("no assignment of pages leaves page 0 free")
    lse = torch.empty(p.q.shape[:2], device=DEV)
    whole = lib.paged_attention(p.q, p.cache, p.batch, causal=causal, window=window, lse=lse)
    p.check(whole, lse, causal=causal, window=window)
    table = p.table.clone()
    gone = torch.ones(p.cache.n_pages, dtype=torch.bool, device=DEV)
    gone[live.long()] = False
    for i, (b, k) in enumerate(released(p)):
        table[b, :k] = (-1, 1 << 30, 0)[i]
    assert any(k for _, k in released(p))
    for name in ("k", "v"):
        t = getattr(p.cache, name)
        if fmt == "bf16":
            t[gone] = math.inf
        else:
            t.view(torch.uint8)[gone] = 0x7F
            getattr(p.cache, name + "_scale")[gone] = math.inf
    out = lib.paged_attention(p.q, p.cache, lib.paged_batch(table, p.kv_len, p.cu_q), causal=causal, window=window)
    assert lib.poll_status() == 0
    assert torch.equal(out, whole)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_a_released_page_inside_the_window_is_still_reported(lib, fmt):
    p = Paged(lib, [(1, 300)], 4, 2, 64, 16, fmt)
    table = p.table.clone()
    table[0, (300 - 40) // 16] = -1
    lib.paged_attention(p.q, p.cache, lib.paged_batch(table, p.kv_len, p.cu_q), window=40)
    assert lib.poll_status() == 7
