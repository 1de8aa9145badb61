"""The loss call's refusals of a gradient that lies over what it is computed from (no GPU: nothing is launched)."""

import ctypes

import pytest

ALIGNED = 1 << 20
INVALID, WORKSPACE = 1, 4
M, H, V = 10, 64, 1000


@pytest.fixture(scope="module")
def L():
    from rank_mlp_gb300 import binding, build
    build.build()
    return binding.load()


# dx is 1280 bytes long, x too, W 128,000
@pytest.mark.parametrize("dx,code", [
    (ALIGNED, INVALID), (ALIGNED + 128, INVALID), (ALIGNED - 128, INVALID), (ALIGNED + 1264, INVALID), (ALIGNED - 1264, INVALID),
    (2 * ALIGNED, INVALID), (2 * ALIGNED + 127984, INVALID), (2 * ALIGNED - 16, INVALID),
    (ALIGNED + 1280, WORKSPACE), (ALIGNED - 1280, WORKSPACE), (2 * ALIGNED + 128000, WORKSPACE), (2 * ALIGNED - 1280, WORKSPACE),
])
def test_dx_over_an_input_is_refused(L, dx, code):
    """(Those that pass are answered by the workspace's size, which is looked at last.)"""
    from rank_mlp_gb300 import binding
    o = binding.LoraCe(1.0, 0.0, 0.0, 1, -100)
    before = L.lora_launch_count()
    assert L.lora_linear_ce(M, H, V, ALIGNED, 2 * ALIGNED, 4 * ALIGNED, ctypes.addressof(o), 5 * ALIGNED, None, 6 * ALIGNED, dx,
                            7 * ALIGNED, 256, None) == code
    assert L.lora_launch_count() == before
