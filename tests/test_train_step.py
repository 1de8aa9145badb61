"""A training step through the library's norm, projections, rotary positions, loss and clipping together
(examples/train_block.py), against the same step in 64 bits; and the same calls in a captured graph."""

import os
import sys

import pytest
import torch

from serving_ref import rotate64
from train_ref import BF16, DEV, rnd, within

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


class Rotate64(torch.autograd.Function):
    @staticmethod
    def forward(ctx, t, rope):
        ctx.rope = rope
        return rotate64(t, rope)[0]

    @staticmethod
    def backward(ctx, d):
        return rotate64(d, ctx.rope, True)[0], None


def loss64(block, lin, x, labels, rope):
    """The block's loss in 64 bits; lin: its projections in 64 bits."""
    batch, seq, hidden = x.shape
    proj = lambda t, n: t @ lin[n][0].T + block.s * (t @ lin[n][1].T) @ lin[n][2].T  # noqa: E731
    norm = lambda t, w: t * (t.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * w.double()  # noqa: E731
    n1 = norm(x, block.norms[0])
    heads = lambda t, n: t.reshape(batch * seq, n, block.head_dim)  # noqa: E731
    per = lambda t, n: t.reshape(batch, seq, n, block.head_dim).transpose(1, 2)  # noqa: E731
    q = per(Rotate64.apply(heads(proj(n1, "q"), block.heads_q), rope), block.heads_q)
    k = per(Rotate64.apply(heads(proj(n1, "k"), block.heads_kv), rope), block.heads_kv)
    v = per(proj(n1, "v"), block.heads_kv)
    group = block.heads_q // block.heads_kv
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    score = (q @ k.transpose(2, 3)) * block.head_dim ** -0.5
    hidden_ = torch.ones(seq, seq, dtype=torch.bool, device=x.device).triu(1)
    a = torch.softmax(score.masked_fill(hidden_, float("-inf")), -1) @ v
    stream = x + proj(a.transpose(1, 2).reshape(batch, seq, -1), "o")
    n2 = norm(stream, block.norms[1])
    g, u = proj(n2, "gate"), proj(n2, "up")
    n3 = norm(stream + proj(torch.nn.functional.silu(g) * u, "down"), block.norms[2])
    z = n3 @ block.head.double().T
    return torch.nn.functional.cross_entropy(z.reshape(-1, z.shape[-1]), labels.reshape(-1))


def leaves64(block):
    return {n: (w.double(), a.detach().double().requires_grad_(), b.detach().double().requires_grad_())
            for n, (w, a, b) in block.lin.items()}


@pytest.mark.parametrize("batch,seq,hide", [(1, 1, 0), (2, 33, 8), (3, 64, 20)])
def test_step_matches_64_bits(lib, batch, seq, hide):
    """Between x and the loss a value is rounded to bf16 some fifteen times, each off by 2^-9 rms at most, and a
    gradient comes back through as many again: sqrt(30) * 2^-9 = 1.1e-2 of a tensor's norm, doubled for the paths
    on which they add up.  Q and K get their gradients through the scores', ds = p (dp - sum p dp): where the two
    terms cancel (one key: ds is 0) what remains is their rounding, 2^-8 of |do| |v|, which reaches q as
    2^-8 |do| |v| |k| / sqrt(d).  With |v| and |k| near sqrt(d), as here, that is 2^-8 sqrt(d) of |do|, v's gradient."""
    import train_block
    block = train_block.Block(128, 344, 4, 2, 64, 1003, device=DEV, seed=3)
    x = rnd(batch, seq, 128, seed=1).requires_grad_()
    labels = torch.randint(0, 1003, (batch, seq), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5))
    labels[:, :hide] = -100
    rope = train_block.rope_of(batch, seq, 64, DEV)
    loss = block.loss(x, labels, rope)
    loss.backward()
    lin, x64 = leaves64(block), x.detach().double().requires_grad_()
    want = loss64(block, lin, x64, labels, rope)
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 2.2e-2 * float(want.detach())

    def close(g, r, n, slack=0.0):
        err = float((g.double() - r).norm())
        assert err <= 2.2e-2 * float(r.norm()) + slack, f"{n}: {err:.2e} of {float(r.norm()):.2e}"
    close(x.grad, x64.grad, "x")
    for n, (w, a, b) in block.lin.items():
        assert w.grad is None
        for k, (got, name) in enumerate(((a, "A_"), (b, "B_"))):
            close(got.grad, lin[n][k + 1].grad, name + n, BF16 * 8 * float(lin["v"][k + 1].grad.norm()) if n in "qk" else 0.0)
    # clipping those gradients, all together
    grads = [p.grad for p in block.adapters]
    before = [g.clone() for g in grads]
    full = sum(float(g.double().square().sum()) for g in before) ** 0.5
    norm = lib.clip_grad_norm(grads, 0.5 * full)
    assert abs(float(norm) - full) <= 1e-5 * full
    for g, b in zip(grads, before):
        within(g, b.double() * (0.5 * full / (full + 1e-6)), (BF16 + 1e-5) * b.double().abs() + 1e-40)
    assert lib.poll_status() == 0


def test_example_steps(lib):
    """The example's step: gradients are consumed, adapters move by lr times the clipped gradients."""
    import train_block
    block = train_block.Block(128, 344, 4, 2, 64, 1003, device=DEV, seed=3)
    x, rope = rnd(2, 16, 128, seed=1), train_block.rope_of(2, 16, 64, DEV)
    labels = torch.randint(0, 1003, (2, 16), device=DEV)
    before = [p.detach().clone() for p in block.adapters]
    block.loss(x, labels, rope).backward()
    grads = [p.grad.clone() for p in block.adapters]
    for p in block.adapters:
        p.grad = None
    full = float(lib.grad_norm(grads))
    loss, norm = train_block.step(block, x, labels, rope, max_norm=0.25 * full, lr=0.5)
    assert float(norm) == full and bool(loss.isfinite())
    for p, b, g in zip(block.adapters, before, grads):
        assert p.grad is None
        want = b.double() - 0.5 * 0.25 * g.double()
        within(p, want, 2 * BF16 * (b.double().abs() + g.double().abs()) + 1e-30)
    assert lib.poll_status() == 0


def test_a_step_of_calls_in_a_graph(lib):
    """Norm, MLP, norm, loss and gradients, clipping, captured once and replayed on other tokens and labels."""
    h, i, V, M = 128, 344, 1003, 96
    lin = lambda s, a, b: (rnd(a, b, seed=s, scale=b ** -0.5), rnd(8, b, seed=s + 1, scale=b ** -0.5),  # noqa: E731
                           rnd(a, 8, seed=s + 2, scale=0.1))
    gate, up, down = lin(1, i, h), lin(4, i, h), lin(7, h, i)
    w1, w2, head = rnd(h, seed=10), rnd(h, seed=11), rnd(V, h, seed=12, scale=h ** -0.5)
    x, y = rnd(M, h, seed=13), torch.randint(0, V, (M,), device=DEV)

    def step():
        n1, s1, r1 = lib.rms_norm(x, w1, training=True)
        m, saved = lib.mlp_forward(n1, gate, up, down, 2.0)
        n2, s2, r2 = lib.rms_norm(m, w2, residual=x, training=True)
        total, loss, lse, dn2 = lib.linear_cross_entropy(n2, head, y)
        ds2, dw2 = lib.rms_norm_backward(dn2, s2, w2, r2)
        g = lib.mlp_backward(n1, gate, up, down, 2.0, "swiglu", saved, ds2)
        dx, dw1 = lib.rms_norm_backward(g["dx"], s1, w1, r1, ds=ds2)
        grads = [g[k] for k in sorted(g) if k != "dx"] + [dw1, dw2]
        return [total, loss, dx, lib.clip_grad_norm(grads, 0.05), *grads]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    for k in range(3):
        torch.cuda.synchronize()
        x.copy_(rnd(M, h, seed=40 + k))
        y.copy_(torch.randint(0, V, (M,), device=DEV))
        y[::k + 2] = -100
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert lib.poll_status() == 0
