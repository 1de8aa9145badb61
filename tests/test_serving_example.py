"""examples/serve_block.py: a LoRA attention block that prefills in chunks and decodes over
the paged cache, against the 64-bit oracle's projections, rotation and attention computed
for whole sequences at once; and the attention kernels' bounded waits."""

import os
import sys

import numpy as np
import pytest
import torch

from helpers import f64
from serving_ref import DEV, Paged, attention64, rotate64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,tol", [("bf16", 1e-2), ("int8", 2e-2), ("fp8", 8e-2)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_chunked_prefill_and_decode_match_the_oracle(lib, fmt, tol, layout):
    """Relative Frobenius error of each sequence's outputs.  The bf16 chain rounds q, k, v, the
    attention and the result (five roundings of 2^-9 rms at most, 1e-2 with room, as for the
    projections alone).  An 8-bit cache adds its own: half an int8 step is 0.4% of a row's
    largest feature (1.5% of a normal row's rms, half of it uniform: 0.9%), an e4m3 code is
    within 2^-4, 3.6% rms for K and for V."""
    import oracle
    import serve_block
    hidden, hq, hk, dim = 256, 8, 2, 64
    block = serve_block.Block(hidden, hq, hk, dim, device=DEV, seed=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    prompts = [torch.randn(n, hidden, generator=g, device=DEV).to(torch.bfloat16) for n in (70, 1, 150)]
    steps = 3
    outs = serve_block.run(block, prompts, steps, fmt, chunk=64, page_size=16, layout=layout)
    cos, sin = lib.rope_table(160, dim, device=DEV)
    for p, out in zip(prompts, outs):
        n = p.shape[0] + steps
        assert out.shape == (n, hidden)
        # the inputs as the block saw them: the prompt, then its own outputs
        x = torch.cat([p, out[p.shape[0] - 1:n - 1]])
        lin = lambda t, l: torch.from_numpy(oracle.lora_linear(f64(t), *(f64(w) for w in l), block.s)).to(DEV)  # noqa: E731
        q, k, v = (lin(x, l).view(n, h, dim) for l, h in ((block.q, hq), (block.k, hk), (block.v, hk)))
        rope = {"cos": cos, "sin": sin, "pos": torch.arange(n, device=DEV), "layout": layout}
        a, _, _, _ = attention64(rotate64(q, rope)[0], rotate64(k, rope)[0], v, 0, dim ** -0.5)
        ref = oracle.lora_linear(a.reshape(n, -1).cpu().numpy(), *(f64(w) for w in block.o), block.s)
        err = np.linalg.norm(f64(out) - ref) / np.linalg.norm(ref)
        assert err <= tol, f"{fmt}: {err:.2e}"


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("lengths,hq,hk,dim", [([(1, 500), (1, 40)], 8, 2, 128), ([(40, 500)], 8, 4, 64),
                                               ([(300, 500)], 8, 2, 128), ([(100, 300)], 4, 4, 256)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(lib, lengths, hq, hk, dim, fmt):
    """The failure-path hook leaves the first pipeline stage of every block empty: the bounded
    waits expire, the kernel leaves, the status word says so."""
    p = Paged(lib, lengths, hq, hk, dim, 32, fmt)
    lib.paged_attention(p.q, p.cache, p.batch)
    torch.cuda.synchronize()
    assert lib.poll_status() == 0
    try:
        lib.set_wait_timeout(20_000_000)
        lib.test_expire_waits(1)
        lib.paged_attention(p.q, p.cache, p.batch)
        torch.cuda.synchronize()
        assert lib.poll_status() == 6
    finally:
        lib.test_expire_waits(0)
        lib.set_wait_timeout(0)
    out = lib.paged_attention(p.q, p.cache, p.batch)
    p.check(out)
    assert lib.poll_status() == 0
