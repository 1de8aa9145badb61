"""The serving calls of the binding refuse tensors that do not all lie on the current device,
before anything reaches the library.  Pretended devices and a pretended library: no GPU."""

import types

import pytest
import torch


class On(torch.Tensor):
    """A host tensor that says it is on a GPU."""

    @staticmethod
    def make(index, *shape, dtype=torch.bfloat16):
        t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
        t.index = index
        return t

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index


@pytest.fixture
def calls(monkeypatch):
    from rank_mlp_gb300 import binding as b
    seen = []

    def entry(name):
        def f(*a):
            seen.append(name)
            return 0
        return f
    monkeypatch.setattr(b, "_LIB", types.SimpleNamespace(
        **{n: entry(n) for n in ("lora_rotary", "lora_kv_append", "lora_kv_read", "lora_paged_attention",
                                 "lora_paged_attention_workspace_bytes")}))
    monkeypatch.setattr(b, "_call", lambda t, n, ws: (0, 256, 256))
    monkeypatch.setattr(b, "_current_device", lambda: 0, raising=False)
    return types.SimpleNamespace(b=b, seen=seen)


I32, F32, I64 = torch.int32, torch.float32, torch.int64
TENSORS = dict(
    q=((6, 4, 64),), k=((6, 2, 64),), v=((6, 2, 64),), q_out=((6, 4, 64),), k_out=((6, 2, 64),),
    cos=((9, 32), F32), sin=((9, 32), F32), pos=((6,), I32), slots=((6,), I64),
    ck=((5, 2, 16, 64), torch.int8), cv=((5, 2, 16, 64), torch.int8), ks=((5, 2, 16), F32), vs=((5, 2, 16), F32),
    table=((3, 2), I32), kv_len=((3,), I32), cu=((4,), I32), out=((6, 4, 64),), lse=((6, 4), F32),
    ws=((1 << 12,), torch.uint8))


def rope(t):
    return {n: t[n] for n in ("cos", "sin", "pos")}


def cache(b, t):
    return b.KVCache(t["ck"], t["cv"], t["ks"], t["vs"])


CALLS = {
    "rotary": (("q", "k", "q_out", "k_out", "cos", "sin", "pos", "ws"), lambda b, t: b.rotary(
        t["q"], t["k"], rope=rope(t), q_out=t["q_out"], k_out=t["k_out"], ws=t["ws"])),
    "kv_append": (("q", "k", "v", "q_out", "slots", "cos", "sin", "pos", "ck", "cv", "ks", "vs", "ws"),
                  lambda b, t: b.kv_append(cache(b, t), t["k"], t["v"], t["slots"], q=t["q"], rope=rope(t),
                                           q_out=t["q_out"], ws=t["ws"])),
    "kv_read": (("table", "cu", "ck", "cv", "ks", "vs", "ws"),
                lambda b, t: b.kv_read(cache(b, t), t["table"], t["cu"], 0, ws=t["ws"])),
    "paged_attention": (("q", "table", "kv_len", "cu", "ck", "cv", "ks", "vs", "out", "lse", "ws"),
                        lambda b, t: b.paged_attention(t["q"], cache(b, t), b.paged_batch(t["table"], t["kv_len"], t["cu"]),
                                                       out=t["out"], lse=t["lse"], ws=t["ws"])),
}


def tensors(elsewhere=None, index=0):
    return {n: On.make(1 if n == elsewhere else index, *a[0], **(dict(dtype=a[1]) if len(a) > 1 else {}))
            for n, a in TENSORS.items()}


@pytest.mark.parametrize("name", CALLS)
def test_one_device_reaches_the_library(calls, name):
    CALLS[name][1](calls.b, tensors())
    assert calls.seen[-1] == "lora_" + name


@pytest.mark.parametrize("name,elsewhere", [(n, t) for n, (ts, _) in CALLS.items() for t in ts])
def test_a_tensor_on_another_device_is_refused(calls, name, elsewhere):
    with pytest.raises(ValueError, match="device"):
        CALLS[name][1](calls.b, tensors(elsewhere))
    assert "lora_" + name not in calls.seen


@pytest.mark.parametrize("name", CALLS)
def test_tensors_off_the_current_device_are_refused(calls, name):
    with pytest.raises(ValueError, match="device"):
        CALLS[name][1](calls.b, tensors(index=2))
    assert "lora_" + name not in calls.seen
