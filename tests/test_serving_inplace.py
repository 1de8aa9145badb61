"""lora_kv_append with yq == q, where a lane's partner features lie in pieces that other lanes
of the row write: every format, rotations that are and are not a multiple of 16."""

import pytest
import torch

from serving_ref import DEV, rope_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("dim,rot,layout", [(64, 20, "half"), (64, 64, "half"), (128, 20, "half"), (128, 126, "half"),
                                            (256, 250, "half"), (256, 128, "half"), (128, 22, "interleaved"),
                                            (256, 250, "interleaved")])
@pytest.mark.parametrize("tokens,hq,hk", [(1, 4, 1), (333, 6, 2), (2000, 32, 8)])
def test_append_q_in_place(lib, fmt, dim, rot, layout, tokens, hq, hk):
    g = torch.Generator(device=DEV).manual_seed(rot)
    q, k, v = (torch.randn(tokens, h, dim, generator=g, device=DEV).to(torch.bfloat16) for h in (hq, hk, hk))
    rope = rope_inputs(tokens, rot, layout)
    slots = torch.arange(tokens, device=DEV)
    caches = [lib.kv_cache(-(-tokens // 16), 16, hk, dim, fmt, device=DEV) for _ in range(2)]
    want = lib.kv_append(caches[0], k, v, slots, q=q, rope=rope)
    assert torch.equal(want, lib.rotary(q, rope=rope))
    own = q.clone()
    assert lib.kv_append(caches[1], k, v, slots, q=own, rope=rope, q_out=own) is own
    assert torch.equal(own, want)
    for n in ("k", "v"):
        assert torch.equal(getattr(caches[0], n).view(torch.uint8), getattr(caches[1], n).view(torch.uint8))
    assert lib.poll_status() == 0
