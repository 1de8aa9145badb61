"""The refusals of the norm, loss and clipping calls on the host (no GPU): every bad argument is answered
with its status before anything is launched, and tensors off the current device do not reach the library.

Only calls that validation rejects are made on the library, so none reaches a CUDA runtime function."""

import ctypes
import types

import pytest
import torch

from test_serving_devices import On

ALIGNED = 1 << 20          # a 256-byte aligned non-null address; never dereferenced
INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from rank_mlp_gb300 import binding, build
    build.build()
    return binding.load()


def _b():
    from rank_mlp_gb300 import binding
    return binding


KEPT = []                  # structures passed by address live until the session ends


def at(s):
    KEPT.append(s)
    return None if s is None else ctypes.addressof(s)


def heads(data=ALIGNED, heads=1, ts=1024, hs=1024):
    return _b().LoraHeads(data, heads, ts, hs)


@pytest.fixture
def nothing_is_launched(L):
    before = L.lora_launch_count()
    yield
    assert L.lora_launch_count() == before


@pytest.mark.usefixtures("nothing_is_launched")
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(x=None), INVALID), (dict(x=dict(data=None)), INVALID), (dict(w=None), INVALID),
    (dict(y=None), INVALID), (dict(dim=0), INVALID), (dict(dim=-8), INVALID), (dict(dim=1020), ALIGNMENT),
    (dict(dim=32776), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED), (dict(M=1 << 30, x=dict(heads=4)), UNSUPPORTED),
    (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID), (dict(offset=INF), INVALID), (dict(fmt=2), INVALID),
    (dict(fmt=1), INVALID), (dict(fmt=0, sc=ALIGNED), INVALID),                   # a scale where none belongs
    (dict(res=None), INVALID), (dict(total=None), INVALID),                       # a sum without a residual
    (dict(res=dict(heads=2)), INVALID), (dict(total=dict(heads=2)), INVALID), (dict(total=dict(ts=8)), INVALID),
    (dict(x=dict(data=ALIGNED + 2)), ALIGNMENT), (dict(x=dict(ts=1020)), ALIGNMENT), (dict(x=dict(ts=-8)), INVALID),
    (dict(w=ALIGNED + 8), ALIGNMENT), (dict(y=ALIGNED + 8), ALIGNMENT), (dict(rstd=ALIGNED + 2), ALIGNMENT),
    (dict(ws=None), INVALID), (dict(ws=ALIGNED + 16), ALIGNMENT), (dict(ws_bytes=255), WORKSPACE),
])
def test_norm_refuses(L, kw, code):
    v = {n: (None if n in kw and kw[n] is None else heads(**kw.get(n, {}))) for n in ("x", "res", "total")}
    assert L.lora_rms_norm(kw.get("M", 10), kw.get("dim", 1024), at(v["x"]), at(v["res"]), kw.get("w", ALIGNED),
                           kw.get("offset", 0.0), kw.get("eps", 1e-6), kw.get("fmt", 0), at(v["total"]),
                           kw.get("y", ALIGNED), kw.get("sc"), kw.get("rstd"), kw.get("ws", ALIGNED),
                           kw.get("ws_bytes", 256), None) == code


@pytest.mark.usefixtures("nothing_is_launched")
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(dy=None), INVALID), (dict(s=None), INVALID), (dict(s=dict(data=None)), INVALID),
    (dict(w=None), INVALID), (dict(rstd=None), INVALID), (dict(dx=None), INVALID), (dict(dim=1020), ALIGNMENT),
    (dict(dim=32776), UNSUPPORTED), (dict(dy=dict(heads=2)), INVALID), (dict(ds=dict(heads=2)), INVALID),
    (dict(offset=NAN), INVALID), (dict(dy=dict(data=ALIGNED + 8)), ALIGNMENT), (dict(ds=dict(ts=4)), ALIGNMENT),
    (dict(dx=ALIGNED + 8), ALIGNMENT), (dict(dw=ALIGNED + 1), ALIGNMENT), (dict(ws=None), INVALID),
    (dict(ws_bytes=256), WORKSPACE), (dict(ws=ALIGNED + 16), ALIGNMENT),
])
def test_norm_backward_refuses(L, kw, code):
    v = {n: (None if n in kw and kw[n] is None else heads(**kw.get(n, {}))) for n in ("dy", "s", "ds")}
    need = L.lora_rms_norm_workspace_bytes(10, 1, 1024)
    assert need > 256
    assert L.lora_rms_norm_backward(kw.get("M", 10), kw.get("dim", 1024), at(v["dy"]), at(v["s"]), kw.get("w", ALIGNED),
                                    kw.get("offset", 0.0), kw.get("rstd", ALIGNED), at(v["ds"]), kw.get("dx", ALIGNED),
                                    kw.get("dw", ALIGNED), kw.get("ws", ALIGNED), kw.get("ws_bytes", need), None) == code


def test_norm_workspace_query(L):
    q = L.lora_rms_norm_workspace_bytes
    assert q(-1, 1, 64) == 0 and q(1, 0, 64) == 0 and q(1, 1, 60) == 0 and q(1, 1, 40000) == 0
    assert q(1 << 30, 1, 4096) == q(1 << 20, 1, 4096) > q(10, 1, 4096) > 256


@pytest.mark.usefixtures("nothing_is_launched")
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(h=0), INVALID), (dict(V=0), INVALID), (dict(h=60), ALIGNMENT), (dict(M=1 << 31), UNSUPPORTED),
    (dict(V=1 << 31), UNSUPPORTED), (dict(V=(1 << 24) + 1), UNSUPPORTED), (dict(h=1 << 31), UNSUPPORTED), (dict(x=None), INVALID), (dict(W=None), INVALID),
    (dict(labels=None), INVALID), (dict(opts=None), INVALID), (dict(total=None), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(softcap=-1.0), INVALID), (dict(softcap=NAN), INVALID),
    (dict(softcap=1e-45), INVALID), (dict(softcap=3e38), INVALID), (dict(smoothing=-0.1), INVALID), (dict(smoothing=1.0), INVALID),
    (dict(smoothing=NAN), INVALID), (dict(reduction=2), INVALID), (dict(dx=ALIGNED + (1 << 12), x=ALIGNED + (1 << 12)), INVALID),
    (dict(x=ALIGNED + 8), ALIGNMENT), (dict(W=ALIGNED + 2), ALIGNMENT), (dict(dx=ALIGNED + 8), ALIGNMENT),
    (dict(labels=ALIGNED + 4), ALIGNMENT), (dict(loss=ALIGNED + 2), ALIGNMENT), (dict(total=ALIGNED + 1), ALIGNMENT),
    (dict(ws=None), INVALID), (dict(ws=ALIGNED + 16), ALIGNMENT), (dict(ws_bytes=1 << 16), WORKSPACE),
])
def test_cross_entropy_refuses(L, kw, code):
    o = _b().LoraCe(kw.get("scale", 1.0), kw.get("softcap", 0.0), kw.get("smoothing", 0.0), kw.get("reduction", 1), -100)
    opts = None if "opts" in kw else at(o)
    need = L.lora_linear_ce_workspace_bytes(10, 64, 1000, at(_b().LoraCe(1.0, 0.0, 0.1, 1, -100)), 1)
    assert need > 1 << 16
    assert L.lora_linear_ce(kw.get("M", 10), kw.get("h", 64), kw.get("V", 1000), kw.get("x", ALIGNED),
                            kw.get("W", 2 * ALIGNED), kw.get("labels", ALIGNED), opts, kw.get("loss", ALIGNED), None,
                            kw.get("total", ALIGNED), kw.get("dx", 3 * ALIGNED), kw.get("ws", ALIGNED),
                            kw.get("ws_bytes", need), None) == code


def test_cross_entropy_workspace_is_bounded_by_pieces(L):
    """It grows with the tokens by x's own size and a few words each, not by the logits."""
    o = _b().LoraCe(1.0, 0.0, 0.0, 1, -100)
    q = lambda M, dx=1, V=131072, opts=o: L.lora_linear_ce_workspace_bytes(M, 1024, V, at(opts), dx)  # noqa: E731
    a, b = q(1 << 16), q(1 << 18)
    assert 0 < b - a <= (3 << 16) * (2 * 1024 + 64) + (1 << 24)
    assert b < (1 << 30) + (1 << 28) + (1 << 18) * (2 * 1024 + 64) + (1 << 24)
    assert q(1 << 18, 0) < (1 << 28) + (1 << 18) * (2 * 1024 + 64) + (1 << 24)
    # a small vocabulary: the product's f32 sums bound the piece
    a, b = q(1 << 18, V=1000), q(1 << 20, V=1000)
    assert 0 < b - a <= (3 << 18) * (2 * 1024 + 64) + (1 << 24) and a < (1 << 31) + (1 << 28) + (1 << 18) * (2 * 1024 + 64)
    assert q(16) < 1 << 28 and q(0) > 0 and q(-1) == 0 and q(16, V=0) == 0
    assert q(16, opts=_b().LoraCe(1.0, -1.0, 0.0, 1, -100)) == 0


@pytest.mark.usefixtures("nothing_is_launched")
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(h=0), INVALID), (dict(x=None), INVALID), (dict(g=None), INVALID), (dict(y=None), INVALID),
    (dict(stride=2), INVALID), (dict(stride=-1), INVALID), (dict(M=1 << 31), UNSUPPORTED), (dict(h=1 << 31), UNSUPPORTED),
    (dict(h=60), ALIGNMENT), (dict(x=ALIGNED + 8), ALIGNMENT), (dict(y=ALIGNED + 2), ALIGNMENT), (dict(g=ALIGNED + 2), ALIGNMENT),
    (dict(ws=None), INVALID), (dict(ws=ALIGNED + 16), ALIGNMENT), (dict(ws_bytes=255), WORKSPACE),
])
def test_scale_rows_refuses(L, kw, code):
    assert L.lora_scale_rows(kw.get("M", 4), kw.get("h", 64), kw.get("x", ALIGNED), kw.get("g", ALIGNED), kw.get("stride", 1),
                             kw.get("y", ALIGNED), kw.get("ws", ALIGNED), kw.get("ws_bytes", 256), None) == code


def tensors(*specs):
    arr = (_b().LoraTensor * max(1, len(specs)))()
    for i, s in enumerate(specs):
        arr[i] = _b().LoraTensor(*s)
    return arr


GOOD = (ALIGNED, 100, 0)


@pytest.mark.usefixtures("nothing_is_launched")
@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(g=None), INVALID), (dict(g=[(None, 4, 0)]), INVALID), (dict(g=[(ALIGNED, -1, 0)]), INVALID),
    (dict(g=[(ALIGNED, 4, 2)]), INVALID), (dict(norm=None), INVALID), (dict(kind=2), INVALID), (dict(n=(1 << 20) + 1), UNSUPPORTED),
    (dict(g=[(ALIGNED, (1 << 40) + 1, 0)]), UNSUPPORTED), (dict(g=[(ALIGNED, 1 << 40, 0)] * 20), UNSUPPORTED),
    (dict(g=[(ALIGNED + 1, 4, 0)]), ALIGNMENT), (dict(g=[(ALIGNED + 2, 4, 1)]), ALIGNMENT), (dict(norm=ALIGNED + 2), ALIGNMENT),
    (dict(ws=None), INVALID), (dict(ws=ALIGNED + 16), ALIGNMENT), (dict(ws_bytes=256), WORKSPACE),
])
def test_grad_norm_and_clip_refuse(L, kw, code):
    specs = kw.get("g", [GOOD])
    arr = None if specs is None else tensors(*specs)
    n = kw.get("n", 1 if specs is None else len(specs))
    ws = (kw.get("ws", ALIGNED), kw.get("ws_bytes", L.lora_grad_norm_workspace_bytes(max(1, min(n, 20)))))
    assert L.lora_grad_norm(n, at(arr), kw.get("kind", 0), kw.get("norm", ALIGNED), *ws, None) == code
    assert L.lora_clip_grads(n, at(arr), None, kw.get("kind", 0), 1.0, kw.get("norm", ALIGNED), *ws, None) == code


@pytest.mark.usefixtures("nothing_is_launched")
@pytest.mark.parametrize("kw,code", [
    (dict(limit=0.0), INVALID), (dict(limit=-1.0), INVALID), (dict(limit=NAN), INVALID),
    (dict(out=[(ALIGNED, 99, 0)]), INVALID), (dict(out=[(ALIGNED, 100, 1)]), INVALID), (dict(out=[(None, 100, 0)]), INVALID),
    (dict(out=[(ALIGNED + 1, 100, 0)]), ALIGNMENT),
])
def test_clip_refuses(L, kw, code):
    need = L.lora_grad_norm_workspace_bytes(1)
    assert L.lora_clip_grads(1, at(tensors(GOOD)), at(tensors(*kw.get("out", [GOOD]))), 0, kw.get("limit", 1.0), ALIGNED,
                             ALIGNED, need, None) == code


@pytest.mark.usefixtures("nothing_is_launched")
@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(g=None), INVALID), (dict(out=None), INVALID), (dict(ex=0), INVALID), (dict(ex=3), INVALID),
    (dict(ex=65536), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(out=[(ALIGNED, 100, 1)]), INVALID),
    (dict(out=[(ALIGNED, 25, 0)]), INVALID), (dict(limit=0.0), INVALID), (dict(limit=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(sq=None), INVALID), (dict(sq=ALIGNED + 2), ALIGNMENT), (dict(out=[(ALIGNED + 2, 25, 1)]), ALIGNMENT),
    (dict(ws=None), INVALID), (dict(ws=ALIGNED + 16), ALIGNMENT), (dict(ws_bytes=256), WORKSPACE),
])
def test_clip_examples_refuses(L, kw, code):
    g = None if "g" in kw else tensors(GOOD)
    out = None if kw.get("out", 1) is None else tensors(*kw.get("out", [(ALIGNED, 25, 1)]))
    need = L.lora_clip_examples_workspace_bytes(1, 4)
    assert need > 256
    assert L.lora_clip_examples(kw.get("n", 1), at(g), kw.get("ex", 4), at(out), kw.get("limit", 1.0), kw.get("scale", 1.0),
                                kw.get("sq", ALIGNED), 0, kw.get("ws", ALIGNED), kw.get("ws_bytes", need), None) == code


def test_list_workspace_queries(L):
    assert L.lora_grad_norm_workspace_bytes(-1) == 0 and L.lora_grad_norm_workspace_bytes((1 << 20) + 1) == 0
    assert L.lora_grad_norm_workspace_bytes(0) > 256
    assert L.lora_clip_examples_workspace_bytes(3, 0) == 0 and L.lora_clip_examples_workspace_bytes(3, 65536) == 0
    assert L.lora_clip_examples_workspace_bytes(0, 1) > 256


def test_binding_refuses_wrong_tensors(L):
    b = _b()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        b.rms_norm(x, w)                                                          # on the host
    with pytest.raises(ValueError):
        b.linear_cross_entropy(x, torch.zeros(10, 32, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        b.linear_cross_entropy(x, torch.zeros(10, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64), reduction="none")
    with pytest.raises(TypeError):
        b.tensor_list([1.0])
    with pytest.raises(ValueError):
        b.tensor_list([x])


# ------------------------------------------------------------------ devices, on a pretended library

@pytest.fixture
def calls(monkeypatch):
    b = _b()
    seen = []

    def entry(name):
        def f(*a):
            if not name.endswith("_bytes"):
                seen.append(name)
            return 0
        return f
    names = [n for n in b.EXPORTS if any(k in n for k in ("norm", "linear_ce", "clip", "scale_rows"))]
    monkeypatch.setattr(b, "_LIB", types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(b, "_call", lambda t, n, ws: (0, 256, 256))
    monkeypatch.setattr(b, "_current_device", lambda: 0)
    monkeypatch.setattr(b, "torch", types.SimpleNamespace(**{**vars(torch), "empty": lambda *s, dtype=None, device=None: On.make(
        0, tuple(s[0]) if s and isinstance(s[0], tuple) else s, dtype=dtype or torch.float32)}))
    return types.SimpleNamespace(b=b, seen=seen)


F32, I64 = torch.float32, torch.int64
SPECS = dict(x=((6, 64),), w=((64,),), r=((6, 64),), s=((6, 64),), out=((6, 64),), rstd=((6,), F32), ds=((6, 64),),
             dx=((6, 64),), W=((9, 64),), y=((6,), I64), g0=((4, 8),), g1=((4, 3), F32), o0=((4, 8),), o1=((4, 3), F32),
             s0=((8,), F32), s1=((3,), F32), sq=((4,), F32), ws=((4096,), torch.uint8))
CALLS = {
    "rms_norm": (("x", "w", "r", "s", "out", "ws"), lambda b, t: b.rms_norm(
        t["x"], t["w"], residual=t["r"], sum_out=t["s"], out=t["out"], ws=t["ws"])),
    "rms_norm_backward": (("x", "w", "s", "rstd", "ds", "dx", "ws"), lambda b, t: b.rms_norm_backward(
        t["x"], t["s"], t["w"], t["rstd"], ds=t["ds"], dx=t["dx"], ws=t["ws"])),
    "linear_ce": (("x", "W", "y", "dx", "ws"), lambda b, t: b.linear_cross_entropy(t["x"], t["W"], t["y"], dx=t["dx"], ws=t["ws"])),
    "scale_rows": (("x", "rstd", "out", "ws"), lambda b, t: b.scale_rows(t["x"], t["rstd"], out=t["out"], ws=t["ws"])),
    "grad_norm": (("g0", "g1", "ws"), lambda b, t: b.grad_norm([t["g0"], t["g1"]], ws=t["ws"])),
    "clip_grads": (("g0", "g1", "o0", "o1", "ws"), lambda b, t: b.clip_grad_norm(
        [t["g0"], t["g1"]], 1.0, out=[t["o0"], t["o1"]], ws=t["ws"])),
    "clip_examples": (("g0", "g1", "s0", "s1", "sq", "ws"), lambda b, t: b.clip_examples(
        [t["g0"], t["g1"]], 1.0, sq_norms=t["sq"], out=[t["s0"], t["s1"]], ws=t["ws"])),
}


def pretended(elsewhere=None, index=0):
    return {n: On.make(1 if n == elsewhere else index, *a[0], **(dict(dtype=a[1]) if len(a) > 1 else {}))
            for n, a in SPECS.items()}


@pytest.mark.parametrize("name", CALLS)
def test_one_device_reaches_the_library(calls, name):
    CALLS[name][1](calls.b, pretended())
    assert calls.seen == ["lora_" + name]


@pytest.mark.parametrize("name,elsewhere", [(n, t) for n, (ts, _) in CALLS.items() for t in ts])
def test_a_tensor_on_another_device_is_refused(calls, name, elsewhere):
    with pytest.raises(ValueError, match="device"):
        CALLS[name][1](calls.b, pretended(elsewhere))
    assert not calls.seen


@pytest.mark.parametrize("name", CALLS)
def test_tensors_off_the_current_device_are_refused(calls, name):
    with pytest.raises(ValueError, match="device"):
        CALLS[name][1](calls.b, pretended(index=2))
    assert not calls.seen
