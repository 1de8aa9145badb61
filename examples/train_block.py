"""One training step of a LoRA-tuned transformer block under a frozen head: norms, projections, the loss
and the clipping run in the library, attention between Q/K/V and O is PyTorch's.

    x -> norm -> q, k, v -> rotary -> attention -> o -> + x, norm -> MLP -> + , norm -> cross entropy
    loss.backward() -> clip_grad_norm over the adapters -> SGD

    python examples/train_block.py [--steps N]
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from rank_mlp_gb300 import autograd as F  # noqa: E402
from rank_mlp_gb300 import binding as lora  # noqa: E402


class Block:
    """Frozen weights of a block and its head, and the adapters (bf16 leaves that train)."""

    def __init__(self, hidden, inter, heads_q, heads_kv, head_dim, vocab, rank=8, alpha=16.0, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s, sd: (torch.randn(*s, generator=g, device=device) * sd).to(torch.bfloat16)  # noqa: E731
        self.heads_q, self.heads_kv, self.head_dim, self.s = heads_q, heads_kv, head_dim, alpha / rank
        n_q, n_kv = heads_q * head_dim, heads_kv * head_dim
        self.lin = {}
        for name, i, o in (("q", hidden, n_q), ("k", hidden, n_kv), ("v", hidden, n_kv), ("o", n_q, hidden),
                           ("gate", hidden, inter), ("up", hidden, inter), ("down", inter, hidden)):
            self.lin[name] = (rnd(o, i, sd=i ** -0.5), rnd(rank, i, sd=i ** -0.5).requires_grad_(),
                              rnd(o, rank, sd=0.1).requires_grad_())
        self.norms = [(1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(torch.bfloat16) for _ in range(3)]
        self.head = rnd(vocab, hidden, sd=hidden ** -0.5)

    @property
    def adapters(self):
        return [t for _, a, b in self.lin.values() for t in (a, b)]

    def loss(self, x, labels, rope):
        """x [batch, seq, hidden], labels [batch, seq]: the mean loss over the labelled tokens."""
        batch, seq, hidden = x.shape
        lin, heads = self.lin, lambda t, n: t.reshape(batch * seq, n, self.head_dim)  # noqa: E731
        n1 = F.lora_rms_norm(x, self.norms[0])
        q, k, v = F.lora_qkv(n1, lin["q"], lin["k"], lin["v"], self.s)
        q, k = F.lora_rotary(heads(q, self.heads_q), heads(k, self.heads_kv), rope)
        per = lambda t, n: t.reshape(batch, seq, n, self.head_dim).transpose(1, 2)  # noqa: E731
        a = torch.nn.functional.scaled_dot_product_attention(
            per(q, self.heads_q), per(k, self.heads_kv), per(v, self.heads_kv), is_causal=True, enable_gqa=True)
        o = F.lora_linear(a.transpose(1, 2).reshape(batch, seq, -1), lin["o"], self.s)
        n2, stream = F.lora_rms_norm(o, self.norms[1], x)
        m = F.lora_mlp(n2, lin["gate"], lin["up"], lin["down"], self.s)
        n3, _ = F.lora_rms_norm(m, self.norms[2], stream)
        return F.lora_linear_cross_entropy(n3, self.head, labels)


def step(block, x, labels, rope, max_norm=1.0, lr=1e-2):
    """One step; returns (loss, gradient norm), both still on the device."""
    loss = block.loss(x, labels, rope)
    loss.backward()
    grads = [p.grad for p in block.adapters]
    norm = lora.clip_grad_norm(grads, max_norm)
    with torch.no_grad():
        for p, g in zip(block.adapters, grads):
            p.sub_(lr * g)
            p.grad = None
    return loss.detach(), norm


def rope_of(batch, seq, head_dim, device):
    cos, sin = lora.rope_table(seq, head_dim, device=device)
    return {"cos": cos, "sin": sin, "pos": torch.arange(seq, device=device, dtype=torch.int32).repeat(batch), "layout": "half"}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    batch, seq, hidden, dev = 4, 1024, 896, "cuda"
    block = Block(hidden, 4864, 14, 2, 64, 131072, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(batch, seq, hidden, generator=g, device=dev).to(torch.bfloat16)
    labels = torch.randint(0, 131072, (batch, seq), generator=g, device=dev)
    labels[:, :seq // 4] = -100                         # the prompt's tokens
    rope = rope_of(batch, seq, 64, dev)
    for _ in range(3):
        step(block, x, labels, rope)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        loss, norm = step(block, x, labels, rope)
    torch.cuda.synchronize()
    assert lora.poll_status() == 0
    print(f"{batch} x {seq} tokens, {a.steps} steps: {(time.perf_counter() - t) / a.steps * 1e3:.2f} ms a step; loss "
          f"{float(loss):.3f}, gradient norm {float(norm):.3f}")


if __name__ == "__main__":
    main()
