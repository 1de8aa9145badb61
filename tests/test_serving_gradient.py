"""autograd's rotary positions: what is saved, which gradients are computed, q alone, gradients of
gradients.  On the host the library's call is a plain 64-bit rotation; on the GPU it runs."""

import pytest
import torch

from serving_ref import DEV, check_rotated, rope_inputs, rotate64


def _rope(tokens, rot, layout, dev="cpu"):
    g = torch.Generator().manual_seed(rot)
    a = torch.rand(50, rot // 2, generator=g) * 6
    return {"cos": a.cos().to(dev), "sin": a.sin().to(dev), "layout": layout,
            "pos": torch.randint(0, 50, (tokens,), generator=g).to(torch.int32).to(dev)}


@pytest.fixture
def plain(monkeypatch):
    """binding.rotary in plain form on the host; its calls (heads of each input, inverse)."""
    from rank_mlp_gb300 import autograd, binding
    calls = []

    def rotary(q, k=None, *, rope, inverse=False):
        calls.append((q.shape[1], None if k is None else k.shape[1], inverse))
        y = [rotate64(t.detach(), rope, inverse)[0].to(t.dtype) for t in (q, k) if t is not None]
        return tuple(y) if k is not None else y[0]
    monkeypatch.setattr(binding, "rotary", rotary)
    monkeypatch.setattr(autograd, "_bf16", lambda t: t)
    return autograd, calls


def _qk(dtype=torch.float64, need=(True, True), heads=(4, 2), dev="cpu"):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(7, h, 16, generator=g, dtype=torch.float64).to(dtype).to(dev).requires_grad_(n)
            for h, n in zip(heads, need)]


@pytest.mark.parametrize("name", ["pos", "cos", "sin"])
def test_tables_changed_in_place_before_the_backward_are_an_error(plain, name):
    q, k = _qk()
    rope = _rope(7, 16, "half")
    yq, yk = plain[0].lora_rotary(q, k, rope)
    rope[name].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (yq.sum() + yk.sum()).backward()


def test_the_callers_dict_may_change(plain):
    q, k = _qk()
    rope = _rope(7, 16, "interleaved")
    want = rotate64(torch.ones_like(q), rope, True)[0]
    yq, _ = plain[0].lora_rotary(q, k, rope)
    rope.update(pos=torch.zeros(7, dtype=torch.int32), layout="half")
    yq.sum().backward()
    assert torch.allclose(q.grad, want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradients_of_gradients(plain, layout):
    q, k = _qk()
    rope = _rope(7, 12, layout)
    f = lambda a, b: plain[0].lora_rotary(a, b, rope)  # noqa: E731
    assert torch.autograd.gradcheck(f, (q, k))
    assert torch.autograd.gradgradcheck(f, (q, k))


def test_q_alone(plain):
    q, _ = _qk()
    rope = _rope(7, 16, "half")
    f = lambda a: plain[0].lora_rotary(a, None, rope)  # noqa: E731
    assert torch.equal(f(q), rotate64(q.detach(), rope)[0])
    assert torch.autograd.gradcheck(f, (q,)) and torch.autograd.gradgradcheck(f, (q,))


@pytest.mark.parametrize("need,back", [((True, False), (4, None, True)), ((False, True), (2, None, True)),
                                       ((True, True), (4, 2, True))])
def test_only_the_gradients_asked_for(plain, need, back):
    q, k = _qk(need=need)
    rope = _rope(7, 16, "half")
    yq, yk = plain[0].lora_rotary(q, k, rope)
    (yq.sum() + yk.sum()).backward()
    assert plain[1] == [(4, 2, False), back]
    for t, n in ((q, need[0]), (k, need[1])):
        assert (t.grad is not None) == n
        if n:
            assert torch.allclose(t.grad, rotate64(torch.ones_like(t), rope, True)[0])


def test_an_output_that_the_loss_leaves_out(plain):
    q, k = _qk()
    rope = _rope(7, 16, "half")
    plain[0].lora_rotary(q, k, rope)[1].sum().backward()
    assert plain[1][1:] == [(2, None, True)]
    assert q.grad is None or not bool(q.grad.any())
    assert torch.allclose(k.grad, rotate64(torch.ones_like(k), rope, True)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_on_the_gpu(lib, layout):
    from rank_mlp_gb300.autograd import lora_rotary
    q, k = _qk(torch.bfloat16, dev=DEV)
    rope = rope_inputs(7, 16, layout)
    y = lora_rotary(q, None, rope)
    check_rotated(y, q.detach(), rope)
    dy = torch.randn_like(y).detach().requires_grad_()
    g, = torch.autograd.grad(y, q, dy, create_graph=True)
    check_rotated(g.detach(), dy.detach(), rope, inverse=True)
    v = torch.randn_like(g).detach()
    gg, = torch.autograd.grad(g, dy, v)
    check_rotated(gg, v, rope)
    yq, yk = lora_rotary(q, k, rope)
    dk = torch.randn(2, 7, 16, device=DEV).to(torch.bfloat16).transpose(0, 1)       # heads first
    gk, = torch.autograd.grad(yk, k, dk)
    check_rotated(gk, dk, rope, inverse=True)
    yq, _ = lora_rotary(q, k, rope)
    rope["pos"].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(yq, q, torch.ones_like(yq))
