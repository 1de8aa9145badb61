"""The serving entry points' refusals on the host (no GPU): every bad argument is answered
with its status before anything is launched, and the size query follows its rules.

Only calls that validation rejects (or that have nothing to do) are made here, so none
reaches a CUDA runtime function."""

import ctypes

import pytest
import torch

ALIGNED = 1 << 20          # a 256-byte aligned non-null address; never dereferenced
INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    from rank_mlp_gb300 import binding, build
    build.build()
    return binding.load()


def _b():
    from rank_mlp_gb300 import binding
    return binding


def heads(data=ALIGNED, heads=4, ts=1024, hs=128):
    return _b().LoraHeads(data, heads, ts, hs)


def rot(cos=ALIGNED, sin=ALIGNED, pos=ALIGNED, n_pos=100, rot_dim=128, layout=0):
    return _b().LoraRotary(cos, sin, pos, n_pos, rot_dim, layout)


def cache(k=ALIGNED, v=ALIGNED, ks=ALIGNED, vs=ALIGNED, n_pages=8, page=16, heads=4, dim=128, fmt=2):
    return _b().LoraKvCache(k, v, ks, vs, n_pages, page, heads, dim, fmt)


def batch(n=2, table=ALIGNED, width=4, kv=ALIGNED, cu=ALIGNED):
    return _b().LoraPagedBatch(n, table, width, kv, cu)


def at(s):
    return None if s is None else ctypes.addressof(s)


@pytest.fixture(autouse=True)
def nothing_is_launched(L):
    before = L.lora_launch_count()
    yield
    assert L.lora_launch_count() == before


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(q=None), INVALID), (dict(yq=None), INVALID), (dict(r=None), INVALID),
    (dict(q=dict(data=None)), INVALID), (dict(yk=None), INVALID), (dict(dim=0), INVALID),
    (dict(dim=2048), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED), (dict(dim=124), ALIGNMENT),
    (dict(r=dict(rot_dim=130)), INVALID), (dict(r=dict(rot_dim=7)), INVALID), (dict(r=dict(rot_dim=0)), INVALID),
    (dict(r=dict(layout=2)), INVALID), (dict(r=dict(n_pos=0)), INVALID), (dict(r=dict(pos=None)), INVALID),
    (dict(r=dict(cos=None)), INVALID), (dict(r=dict(sin=ALIGNED + 4)), ALIGNMENT),
    (dict(r=dict(pos=ALIGNED + 2)), ALIGNMENT), (dict(r=dict(n_pos=1 << 31)), UNSUPPORTED),
    (dict(q=dict(data=ALIGNED + 2)), ALIGNMENT), (dict(q=dict(ts=1020)), ALIGNMENT), (dict(q=dict(ts=-8)), INVALID),
    (dict(yq=dict(ts=0)), INVALID), (dict(yq=dict(hs=64)), INVALID),          # rows of the output overlap
    (dict(yq=dict(ts=256, hs=128)), INVALID), (dict(yq=dict(heads=5)), INVALID), (dict(yk=dict(heads=5)), INVALID),
    (dict(q=dict(heads=0)), INVALID), (dict(ws=None), INVALID), (dict(ws=ALIGNED + 16), ALIGNMENT),
    (dict(ws_bytes=128), WORKSPACE),
])
def test_rotary_refuses(L, kw, code):
    v = {n: (None if n in kw and kw[n] is None else heads(**kw.get(n, {}))) for n in ("q", "yq", "k", "yk")}
    r = None if "r" in kw and kw["r"] is None else rot(**kw.get("r", {}))
    assert L.lora_rotary(kw.get("M", 10), kw.get("dim", 128), at(v["q"]), at(v["yq"]), at(v["k"]), at(v["yk"]), at(r),
                         0, kw.get("ws", ALIGNED), kw.get("ws_bytes", 256), None) == code


def test_rotary_of_no_tokens(L):
    assert L.lora_rotary(0, 128, at(heads(None)), at(heads(None)), None, None, at(rot(pos=None)), 0, ALIGNED, 256,
                         None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(kind=5), INVALID), (dict(kind=1, factor=0.5), INVALID), (dict(kind=1, factor=float("nan")), INVALID),
    (dict(kind=2, factor=2.0, rot_dim=2), INVALID), (dict(kind=3, factor=2.0), INVALID),
    (dict(kind=3, factor=2.0, original_len=64.0, low=4.0, high=4.0), INVALID),
    (dict(kind=4, factor=2.0, original_len=64.0, low=0.0, high=4.0), INVALID),
    (dict(kind=0, magnitude=-1.0), INVALID), (dict(kind=0, rot_dim=7), INVALID), (dict(kind=0, n_pos=0), INVALID),
    (dict(kind=0, base=0.0), INVALID), (dict(kind=0, cos=ALIGNED + 8), ALIGNMENT),
    (dict(kind=0, n_pos=1 << 31), UNSUPPORTED),
])
def test_scaled_table_refuses(L, kw, code):
    a = dict(factor=1.0, original_len=0.0, low=1.0, high=4.0, magnitude=0.0)
    a.update({k: v for k, v in kw.items() if k in a})
    st = _b().LoraRopeScaling(kw["kind"], a["factor"], a["original_len"], a["low"], a["high"], a["magnitude"])
    assert L.lora_rope_table_scaled(kw.get("cos", ALIGNED), ALIGNED, kw.get("n_pos", 16), kw.get("rot_dim", 64),
                                    kw.get("base", 10000.0), at(st), None) == code
    assert L.lora_rope_table_scaled(ALIGNED, ALIGNED, 16, 64, 10000.0, None, None) == INVALID


CACHE_RULES = [
    (dict(c=None), INVALID), (dict(c=dict(k=None)), INVALID), (dict(c=dict(ks=None)), INVALID),
    (dict(c=dict(n_pages=0)), INVALID), (dict(c=dict(fmt=3)), INVALID), (dict(c=dict(fmt=-1)), INVALID),
    (dict(c=dict(page=8)), UNSUPPORTED), (dict(c=dict(page=48)), UNSUPPORTED), (dict(c=dict(page=512)), UNSUPPORTED),
    (dict(c=dict(dim=96)), UNSUPPORTED), (dict(c=dict(n_pages=1 << 25)), UNSUPPORTED),   # rows past 2^31
    (dict(c=dict(k=ALIGNED + 8)), ALIGNMENT), (dict(c=dict(vs=ALIGNED + 2)), ALIGNMENT),
    (dict(ws=ALIGNED + 16), ALIGNMENT), (dict(ws=None), INVALID), (dict(ws_bytes=128), WORKSPACE),
]


@pytest.mark.parametrize("kw,code", CACHE_RULES + [
    (dict(M=-1), INVALID), (dict(k=None), INVALID), (dict(k=dict(heads=3)), INVALID), (dict(v=dict(heads=5)), INVALID),
    (dict(v=dict(data=ALIGNED + 4)), ALIGNMENT), (dict(slots=None), INVALID), (dict(slots=ALIGNED + 4), ALIGNMENT),
    (dict(r=None), INVALID),                                                 # q without rot
    (dict(r=dict(rot_dim=256)), INVALID), (dict(yq=None), INVALID), (dict(yq=dict(heads=3)), INVALID),
    (dict(yq=dict(ts=8)), INVALID), (dict(M=1 << 31), UNSUPPORTED),
])
def test_append_refuses(L, kw, code):
    v = {n: (None if n in kw and kw[n] is None else heads(**kw.get(n, {}))) for n in ("k", "v", "q", "yq")}
    c = None if "c" in kw and kw["c"] is None else cache(**kw.get("c", {}))
    r = None if "r" in kw and kw["r"] is None else rot(**kw.get("r", {}))
    assert L.lora_kv_append(kw.get("M", 10), at(c), at(v["k"]), at(v["v"]), kw.get("slots", ALIGNED), at(v["q"]),
                            at(v["yq"]), at(r), kw.get("ws", ALIGNED), kw.get("ws_bytes", 256), None) == code


@pytest.mark.parametrize("kw,code", CACHE_RULES + [
    (dict(n=0), INVALID), (dict(total=-1), INVALID), (dict(table=None), INVALID), (dict(width=0), INVALID),
    (dict(cu=None), INVALID), (dict(k=None), INVALID), (dict(k=ALIGNED + 2), ALIGNMENT),
    (dict(cu=ALIGNED + 2), ALIGNMENT), (dict(total=1 << 31), UNSUPPORTED),
])
def test_read_refuses(L, kw, code):
    c = None if "c" in kw and kw["c"] is None else cache(**kw.get("c", {}))
    assert L.lora_kv_read(kw.get("n", 2), kw.get("total", 10), at(c), kw.get("table", ALIGNED), kw.get("width", 4),
                          kw.get("cu", ALIGNED), kw.get("k", ALIGNED), ALIGNED, kw.get("ws", ALIGNED),
                          kw.get("ws_bytes", 256), None) == code


@pytest.mark.parametrize("kw,code", CACHE_RULES + [
    (dict(M=-1), INVALID), (dict(q=None), INVALID), (dict(q=dict(data=None)), INVALID), (dict(hq=6), INVALID),
    (dict(hq=0), INVALID), (dict(q=dict(heads=4)), INVALID), (dict(b=None), INVALID), (dict(b=dict(n=0)), INVALID),
    (dict(b=dict(table=None)), INVALID), (dict(b=dict(kv=None)), INVALID), (dict(b=dict(cu=None)), INVALID),
    (dict(b=dict(width=0)), INVALID), (dict(out=None), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(out=ALIGNED + 8), ALIGNMENT),
    (dict(lse=ALIGNED + 2), ALIGNMENT), (dict(q=dict(hs=130, heads=8)), ALIGNMENT), (dict(M=1 << 31), UNSUPPORTED),
    (dict(b=dict(cu=ALIGNED + 2)), ALIGNMENT), (dict(b=dict(width=1 << 28)), UNSUPPORTED),
])
def test_attention_refuses(L, kw, code):
    q = None if "q" in kw and kw["q"] is None else heads(**{"heads": 8, **kw.get("q", {})})
    c = None if "c" in kw and kw["c"] is None else cache(**kw.get("c", {}))
    b = None if "b" in kw and kw["b"] is None else batch(**kw.get("b", {}))
    need = max(256, L.lora_paged_attention_workspace_bytes(10, 2, 8, at(cache())))
    assert L.lora_paged_attention(kw.get("M", 10), kw.get("hq", 8), at(q), at(c), at(b), kw.get("scale", 0.1), 1,
                                  kw.get("window", 0), kw.get("out", ALIGNED), kw.get("lse"), kw.get("ws", ALIGNED),
                                  kw.get("ws_bytes", need), None) == code


def test_attention_workspace_query(L):
    need = L.lora_paged_attention_workspace_bytes
    assert need(10, 2, 8, at(cache())) >= 256
    assert need(10, 2, 6, at(cache())) == 0 and need(-1, 2, 8, at(cache())) == 0
    assert need(10, 0, 8, at(cache())) == 0 and need(10, 2, 8, at(cache(page=20))) == 0


def test_binding_refuses_wrong_tensors(L):
    """Checks that need no GPU: types, shapes, devices."""
    b = _b()
    cpu = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        b.rotary(cpu, rope={"cos": torch.zeros(4, 32), "sin": torch.zeros(4, 32),
                            "pos": torch.zeros(4, dtype=torch.int32)})
    with pytest.raises(TypeError):
        b._heads([1, 2], "q")
    with pytest.raises(ValueError):
        b.KVCache(torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64))              # f32 pages
    with pytest.raises(ValueError):
        b.KVCache(torch.zeros(2, 2, 16, 64, dtype=torch.int8), torch.zeros(2, 2, 16, 64, dtype=torch.int8))   # no scales
    with pytest.raises(ValueError):
        b.PagedBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                     torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        b.rope_table_scaled(4, 64, scaling=dict(kind="linear", facto=2.0))
