"""Lists of tensors that are kept from call to call, on a pretended library: no GPU."""

import struct
import types

import pytest
import torch

from test_serving_devices import On

F32 = torch.float32


@pytest.fixture
def calls(monkeypatch):
    """The binding over a library that keeps what it was given: (name, its arguments)."""
    from rank_mlp_gb300 import binding as b
    seen = []

    def entry(name):
        def f(*a):
            if not name.endswith("_bytes"):
                seen.append((name, a))
            return 0
        return f
    names = [n for n in b.EXPORTS if any(k in n for k in ("norm", "clip"))]
    monkeypatch.setattr(b, "_LIB", types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(b, "_call", lambda t, n, ws: (0, 256, 256))
    monkeypatch.setattr(b, "_current_device", lambda: 0)
    monkeypatch.setattr(b, "torch", types.SimpleNamespace(**{**vars(torch), "empty": lambda *s, dtype=None, device=None: On.make(
        0, tuple(s[0]) if s and isinstance(s[0], tuple) else s, dtype=dtype or F32)}))
    return types.SimpleNamespace(b=b, seen=seen)


def given(packed):
    """[(address, elements, type)] of a list as the library gets it."""
    v = struct.unpack("=" + "QqQ" * (len(packed) // 24), packed)
    return [tuple(v[i:i + 3]) for i in range(0, len(v), 3)]


def of(*ts):
    return [(t.data_ptr(), t.numel(), {torch.bfloat16: 0, F32: 1}[t.dtype]) for t in ts]


def move(t, *shape):
    """Gives t other memory, as t.data = ... does on a device."""
    t.set_(torch.zeros(*shape, dtype=t.dtype))


@pytest.mark.parametrize("name", ["grad_norm", "clip_grad_norm", "out"])
def test_a_kept_list_follows_its_tensors(calls, name):
    """The library gets the addresses that the tensors have at the call."""
    b = calls.b
    ts, outs = [On.make(0, 40), On.make(0, 7, dtype=F32)], [On.make(0, 40), On.make(0, 7, dtype=F32)]
    kept, out = b.tensor_list(ts), b.tensor_list(outs)

    def call():
        if name == "grad_norm":
            b.grad_norm(kept)
        else:
            b.clip_grad_norm(kept, 1.0, out=out if name == "out" else None)
        a = calls.seen[-1][1]
        return given(a[1]), given(a[2]) if name == "out" else None
    assert call() == (of(*ts), of(*outs) if name == "out" else None)
    first = call()
    assert call() == first
    move(ts[1], 9)
    move(outs[1], 9)
    assert call() == (of(*ts), of(*outs) if name == "out" else None) != first
    ts[0].set_()                                     # nothing is left of it
    outs[0].set_()
    assert call()[0] == of(*ts) and call()[0][0][1] == 0


def test_examples_follow_too(calls, monkeypatch):
    b = calls.b
    monkeypatch.setattr(b, "_together", lambda *ts: None)        # (views of a pretended tensor are on no device)
    g = On.make(0, 4, 8)
    kept = b.tensor_list([g])
    sums, _ = b.clip_examples(kept, 1.0)
    assert sums[0].shape == (8,) and calls.seen[-1][1][2] == 4
    move(g, 3, 5)
    sums, _ = b.clip_examples(kept, 1.0)
    a = calls.seen[-1][1]
    assert given(a[1]) == of(g) and a[2] == 3 and sums[0].shape == (5,)


def test_a_list_that_moved_is_looked_over_again(calls):
    """What a list refuses when it is built it refuses later."""
    b = calls.b
    t = On.make(0, 6, 8)
    kept = b.tensor_list([t])
    t.set_(torch.zeros(8, 6, dtype=torch.bfloat16).t())
    with pytest.raises(ValueError, match="contiguous"):
        b.clip_grad_norm(kept, 1.0)
    u, v = On.make(0, 50), On.make(0, 50)
    kept = b.tensor_list([u, v])
    u.set_(v)
    with pytest.raises(ValueError, match="overlap"):
        b.clip_grad_norm(kept, 1.0)
    assert not calls.seen


def test_memory_that_a_kept_list_knows_is_not_given_away(calls):
    """So an address that is the same is the same memory; until the list follows its tensor."""
    t = On.make(0, 1000)
    kept, old = calls.b.tensor_list([t]), t.data_ptr()
    move(t, 10)
    assert [m.data_ptr() for m in kept._memory] == [old]
    calls.b.grad_norm(kept)
    assert [m.data_ptr() for m in kept._memory] == [t.data_ptr()]


def test_an_output_over_another_gradient_is_refused(calls):
    """out's tensors overlap no gradient but the one in their own place, and that one exactly."""
    b = calls.b
    t = On.make(0, 100)
    part = lambda a, z: as_on(t[a:z])  # noqa: E731

    def as_on(u):
        u.index = 0
        return u
    x, y, z = On.make(0, 30), On.make(0, 30), On.make(0, 30)
    good = [([x, y], [x, y]), ([x, y], [z, y]), ([x, x], [y, z]), ([part(0, 30), part(30, 60)], [part(0, 30), part(60, 90)]),
            ([On.make(0, 0), x], [On.make(0, 0), x])]
    bad = [([x, y], [y, x]), ([x, y], [y, z]), ([x, x], [x, z]), ([part(0, 30)], [part(1, 31)]), ([part(0, 30)], [part(29, 59)]),
           ([part(0, 60), x], [On.make(0, 60), part(59, 89)]), ([x, part(10, 40)], [part(30, 60), y]),
           ([part(0, 5), part(40, 60)], [part(20, 25), part(30, 50)])]
    for grads, out in good + good:
        b.clip_grad_norm(grads, 1.0, out=out)
        b.clip_grad_norm(b.tensor_list(grads), 1.0, out=b.tensor_list(out))
    n = len(calls.seen)
    for grads, out in bad:
        with pytest.raises(ValueError, match="overlap"):
            b.clip_grad_norm(grads, 1.0, out=out)
    assert len(calls.seen) == n
    # a list that has been compared with one is compared with another, and again once either has moved
    out = b.tensor_list([z])
    b.clip_grad_norm([x], 1.0, out=out)
    with pytest.raises(ValueError, match="overlap"):
        b.clip_grad_norm([On.make(0, 30), z], 1.0, out=b.tensor_list([z, y]))
    with pytest.raises(ValueError, match="overlap"):
        b.clip_grad_norm([as_on(z[1:])], 1.0, out=b.tensor_list([as_on(z[:-1])]))
    kept = b.tensor_list([x])
    b.clip_grad_norm(kept, 1.0, out=out)
    z.set_(x.untyped_storage(), 10, (20,))
    with pytest.raises(ValueError, match="overlap"):
        b.clip_grad_norm(kept, 1.0, out=out)
    z.set_(x)
    b.clip_grad_norm(kept, 1.0, out=out)


def test_sums_of_examples_over_their_gradients_are_refused(calls):
    b = calls.b
    g = On.make(0, 4, 20, dtype=F32)
    sq = On.make(0, 4, dtype=F32)
    own = g.view(-1)[40:60]
    over = sq.as_strided((2,), (1,))
    own.index = over.index = 0
    b.clip_examples([g], 1.0, out=[On.make(0, 20, dtype=F32)], sq_norms=sq)
    n = len(calls.seen)
    with pytest.raises(ValueError, match="overlap"):
        b.clip_examples([g], 1.0, out=[own])
    with pytest.raises(ValueError, match="overlap"):
        b.clip_examples([On.make(0, 4, 2, dtype=F32)], 1.0, out=[over], sq_norms=sq)
    assert len(calls.seen) == n


@pytest.mark.parametrize("norm_type", [1.0, 3, 0, -float("inf"), float("nan")])
def test_other_norms_are_refused_by_name(calls, norm_type):
    """An error of the call's arguments, as for all others."""
    b, t = calls.b, On.make(0, 8)
    for call in (lambda: b.grad_norm([t], norm_type=norm_type), lambda: b.clip_grad_norm([t], 1.0, norm_type=norm_type)):
        with pytest.raises(ValueError, match="norm_type"):
            call()
    assert not calls.seen


def test_norm_types_that_there_are(calls):
    b, t = calls.b, On.make(0, 8)
    for norm_type, code in ((2, 0), (2.0, 0), ("inf", 1), (float("inf"), 1)):
        b.grad_norm([t], norm_type=norm_type)
        assert calls.seen[-1][1][2] == code


def test_another_format_of_the_norm_is_refused_by_name(calls):
    b = calls.b
    with pytest.raises(ValueError, match="format"):
        b.rms_norm(On.make(0, 4, 64), On.make(0, 64), format="int8")
    assert not calls.seen
