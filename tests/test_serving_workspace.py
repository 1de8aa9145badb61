"""The cached workspaces and stream capture: what a graph has recorded stays, however large the
calls between its replays are, and its errors are still read."""

import ctypes
import gc
import types
import weakref

import pytest
import torch

from serving_ref import DEV, Paged


@pytest.fixture
def host(monkeypatch):
    """The binding's workspace cache over host memory, on one pretended stream; `.capturing` says
    whether the stream is."""
    from rank_mlp_gb300 import binding as b
    state = types.SimpleNamespace(capturing=False, stream=7, binding=b)
    stream = lambda *a: types.SimpleNamespace(cuda_stream=state.stream)  # noqa: E731
    monkeypatch.setattr(b, "torch", types.SimpleNamespace(
        uint8=torch.uint8, Tensor=torch.Tensor, device=lambda *a: torch.device("cpu"),
        zeros=lambda n, dtype, device: torch.zeros(n, dtype=dtype),
        cuda=types.SimpleNamespace(current_device=lambda: -1, current_stream=stream)))
    monkeypatch.setattr(b, "_capturing", lambda: state.capturing, raising=False)
    monkeypatch.setattr(b, "_WS", {})
    monkeypatch.setattr(b, "_RECORDED", {}, raising=False)

    def poll(ptr, _):
        word = ctypes.c_uint32.from_address(ptr.value)
        code, word.value = word.value, 0
        return code
    monkeypatch.setattr(b, "load", lambda: types.SimpleNamespace(lora_poll_status=poll))
    return state


def test_a_recorded_workspace_outlives_growth(host):
    b = host.binding
    b.workspace(1000, 0)
    host.capturing = True
    recorded = weakref.ref(b.workspace(1000, 0))
    host.capturing = False
    large = b.workspace(5000, 0)
    assert large.numel() >= 5000 and b.workspace(10, 0) is large
    gc.collect()
    assert recorded() is not None, "the buffer that a graph writes to was freed"
    # the next capture records the larger one, and both stay
    host.capturing = True
    assert b.workspace(10, 0) is large
    host.capturing = False
    recorded2, large = weakref.ref(large), None
    b.workspace(9000, 0)
    gc.collect()
    assert recorded() is not None and recorded2() is not None


def test_a_workspace_that_no_graph_recorded_is_freed(host):
    b = host.binding
    first = weakref.ref(b.workspace(1000, 0))
    b.workspace(5000, 0)
    gc.collect()
    assert first() is None


def test_poll_reads_recorded_workspaces_too(host):
    b = host.binding
    host.capturing = True
    recorded = b.workspace(1000, 0)
    host.capturing = False
    b.workspace(5000, 0)
    assert b.poll_status() == 0
    recorded[:4].view(torch.int32)[0] = 7                # a replay reports a bad input
    assert b.poll_status() == 7
    assert b.poll_status() == 0
    recorded[:4].view(torch.int32)[0] = 7
    host.stream = 8                                      # another stream has workspaces of its own
    assert b.poll_status() == 0
    host.stream = 7
    b.workspace(10, 0)[:4].view(torch.int32)[0] = 6
    assert b.poll_status() == 6
    assert b.poll_status() == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_attention_needs_the_same_workspace_at_every_size(dim, fmt):
    from rank_mlp_gb300 import binding as b
    from rank_mlp_gb300 import build
    build.build()
    c = b.LoraKvCache(1 << 20, 1 << 20, 1 << 20, 1 << 20, 8, 16, 4, dim, fmt)
    need = lambda *a: b.load().lora_paged_attention_workspace_bytes(*a, ctypes.addressof(c))  # noqa: E731
    first = need(1, 1, 4)
    assert first > 256
    assert {need(1, 64, 16), need(64, 64, 16), need(256, 64, 16), need(257, 64, 16), need(8192, 4, 64)} == {first}


def _step_and_graph(lib, p, stream):
    with torch.cuda.stream(stream):
        lib.paged_attention(p.q, p.cache, p.batch)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = lib.paged_attention(p.q, p.cache, p.batch)
    return graph, out


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_replays_beside_larger_calls_on_their_stream(lib, fmt):
    p = Paged(lib, [(1, 3000), (1, 40), (1, 700)], 8, 2, 128, 64, fmt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph, out = _step_and_graph(lib, p, s)
    with torch.cuda.stream(s):
        big = Paged(lib, [(2048, 2048)], 8, 2, 128, 64, fmt)
        big.check(lib.paged_attention(big.q, big.cache, big.batch))
        before = lib.workspace(256, DEV).numel()
        lib.workspace(4 * before, DEV)                   # as a larger projection would ask for
        fresh = [torch.full((1 << 20,), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(96)]
        for kv in (3000, 2500, 64):
            p.kv_len[0] = kv
            p.lengths[0] = (1, kv)
            s.synchronize()
            graph.replay()
            s.synchronize()
            p.check(out)
        assert all(bool((f == 0x5A).all()) for f in fresh), "a replay wrote to memory that is not its own"
        p.kv_len[0] = 1 << 28                            # past the table: reported by the replay
        graph.replay()
        assert lib.poll_status() == 7
        assert lib.poll_status() == 0
