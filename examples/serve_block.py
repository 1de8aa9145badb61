"""A LoRA-tuned attention block that answers: prompts of different lengths go through it in
chunks, then every sequence decodes one token at a time, all in one paged K/V cache.

One step is four calls of the library on the current stream:

    qkvo_forward     q, k, v of the step's tokens (frozen weights plus adapters)
    kv_append        q and k rotated, k and v quantised into the cache
    paged_attention  the tokens' attention over everything cached so far
    qkvo_forward     the output projection

    python examples/serve_block.py [--format bf16|fp8|int8] [--steps N]
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from rank_mlp_gb300 import binding as lora  # noqa: E402


class Block:
    """Weights of one attention block: q, k, v and o as (W, A, B) triples (bf16, W frozen)."""

    def __init__(self, hidden, heads_q, heads_kv, head_dim, rank=8, alpha=16.0, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda o, i, sd: (torch.randn(o, i, generator=g, device=device) * sd).to(torch.bfloat16)  # noqa: E731
        lin = lambda i, o: (rnd(o, i, i ** -0.5), rnd(rank, i, i ** -0.5), rnd(o, rank, 0.1))  # noqa: E731
        n_q, n_kv = heads_q * head_dim, heads_kv * head_dim
        self.q, self.k, self.v, self.o = lin(hidden, n_q), lin(hidden, n_kv), lin(hidden, n_kv), lin(n_q, hidden)
        self.heads_q, self.heads_kv, self.head_dim, self.s = heads_q, heads_kv, head_dim, alpha / rank

    def step(self, x, cache, batch, slots, rope):
        """x [tokens, hidden] of the step's sequences -> [tokens, hidden]."""
        p, _ = lora.qkvo_forward(x, self.q, self.k, self.v, None, None, self.s, training=False)
        heads = lambda t, n: t.view(x.shape[0], n, self.head_dim)  # noqa: E731
        q = heads(p["q"], self.heads_q)
        lora.kv_append(cache, heads(p["k"], self.heads_kv), heads(p["v"], self.heads_kv), slots, q=q, rope=rope, q_out=q)
        a = lora.paged_attention(q, cache, batch)
        y, _ = lora.qkvo_forward(None, None, None, None, a.view(x.shape[0], -1), self.o, self.s, training=False)
        return y["o"]


class Sequences:
    """Which pages each sequence owns and how long it is: the host's side of the cache."""

    def __init__(self, count, max_len, page_size, device="cuda"):
        self.page, width = page_size, -(-max_len // page_size)
        self.table = torch.randperm(count * width, device=device).view(count, width).to(torch.int32)
        self.lengths = [0] * count
        self.device = device

    @property
    def n_pages(self):
        return self.table.numel()

    def extend(self, new):
        """Appends new[b] positions to sequence b: (batch, slots, positions) of the step."""
        kv = [a + n for a, n in zip(self.lengths, new)]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        dev = self.device
        pos = torch.cat([torch.arange(a, b, device=dev) for a, b in zip(self.lengths, kv)])
        seq = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev))
        slots = self.table[seq, pos // self.page].long() * self.page + pos % self.page
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        self.lengths = kv
        return lora.paged_batch(self.table, i32(kv), i32(cu)), slots, pos.to(torch.int32)


def run(block, prompts, steps, cache_format="int8", chunk=256, page_size=64, hidden=None, layout="half", scaling=None):
    """Prefills the prompts (a list of [length, hidden] tensors) chunk by chunk, then decodes
    `steps` tokens (a step's output is the next step's input).  Returns the outputs of each
    sequence, [length + steps, hidden]."""
    dev = prompts[0].device
    max_len = max(p.shape[0] for p in prompts) + steps
    seqs = Sequences(len(prompts), max_len, page_size, dev)
    cache = lora.kv_cache(seqs.n_pages, page_size, block.heads_kv, block.head_dim, cache_format, dev)
    cos, sin = lora.rope_table_scaled(max_len, block.head_dim, scaling=scaling, device=dev)
    outs = [[] for _ in prompts]

    def step(parts):
        batch, slots, pos = seqs.extend([p.shape[0] for p in parts])
        y = block.step(torch.cat(parts), cache, batch, slots, {"cos": cos, "sin": sin, "pos": pos, "layout": layout})
        for b, part in enumerate(y.split([p.shape[0] for p in parts])):
            outs[b].append(part)

    for at in range(0, max(p.shape[0] for p in prompts), chunk):
        step([p[at:at + chunk] for p in prompts])       # a prompt that has ended adds no tokens
    for _ in range(steps):
        step([o_last(o) for o in outs])
    assert lora.poll_status() == 0
    return [torch.cat(o) for o in outs]


def o_last(parts):
    return next(p for p in reversed(parts) if p.shape[0])[-1:]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--format", choices=("bf16", "fp8", "int8"), default="int8")
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    hidden, dev = 4096, "cuda"
    block = Block(hidden, 32, 8, 128, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    prompts = [torch.randn(n, hidden, generator=g, device=dev).to(torch.bfloat16) for n in (700, 33, 1500, 256)]
    run(block, prompts, 2, a.format)                    # warm up: workspaces, limits
    torch.cuda.synchronize()
    t = time.perf_counter()
    out = run(block, prompts, a.steps, a.format)
    torch.cuda.synchronize()
    print(f"{sum(p.shape[0] for p in prompts)} prompt tokens in chunks and {a.steps} decode steps of {len(prompts)} "
          f"sequences, {a.format} cache: {(time.perf_counter() - t) * 1e3:.1f} ms; |out| "
          f"{float(out[0].float().abs().mean()):.3f}")


if __name__ == "__main__":
    main()
