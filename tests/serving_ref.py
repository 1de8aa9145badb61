"""Plain 64-bit forms of the serving operators (rotary, paged cache, attention over it),
written from the formulas in include/lora_gb300.h, and the error bounds that the tests
hold the kernels to.

U is bf16's unit roundoff (8 significant bits, ties to even): |bf16(x) - x| <= U |x|.
"""

from __future__ import annotations

import math

import torch

U = 2.0 ** -8
F32 = 2.0 ** -24
DEV = "cuda:0"
TOP = {"int8": 127.0, "fp8": 448.0}


def tables64(n_pos, rot, base=10000.0):
    w = torch.tensor([base ** (-2.0 * c / rot) for c in range(rot // 2)], dtype=torch.float64)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * w
    return a.cos(), a.sin()


def rope_inputs(tokens, rot, layout, seed=0, n_pos=500):
    g = torch.Generator().manual_seed(seed)
    cos, sin = (t.float().to(DEV) for t in tables64(n_pos, rot))
    pos = torch.randint(0, n_pos, (tokens,), generator=g).to(torch.int32).to(DEV)
    return {"cos": cos, "sin": sin, "pos": pos, "layout": layout}


def rotate64(x, rope, inverse=False):
    """(rotated x, the magnitude |a| |cos| + |b| |sin| that its f32 error is relative to)."""
    x = x.double()
    half = rope["cos"].shape[1]
    cos, sin = (rope[n].double()[rope["pos"].long()][:, None] for n in ("cos", "sin"))
    if inverse:
        sin = -sin
    y, mag = x.clone(), x.abs()
    ia = torch.arange(half) if rope["layout"] == "half" else 2 * torch.arange(half)
    ib = ia + (half if rope["layout"] == "half" else 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    mag[..., ia] = a.abs() * cos.abs() + b.abs() * sin.abs()
    mag[..., ib] = b.abs() * cos.abs() + a.abs() * sin.abs()
    return y, mag


def check_rotated(got, x, rope, inverse=False):
    """Two products and a sum in f32 (3 roundings, each at most F32 of the magnitude), one
    rounding to bf16."""
    ref, mag = rotate64(x, rope, inverse)
    err = (got.double() - ref).abs()
    bound = U * ref.abs() + 4 * F32 * mag
    assert bool((err <= bound * 1.001).all()), f"rotation off by {float((err - bound).max()):.3e} over its bound"


def cache_values64(cache, n):
    x = getattr(cache, n)
    x = (x.view(torch.uint8) if x.element_size() == 1 else x).clone().view(x.dtype).double()
    sc = getattr(cache, n + "_scale")
    return x if sc is None else x * sc.double()[..., None]


def attention64(q, k, v, p0, scale, causal=True, window=0):
    """One sequence: q [n, hq, D], k and v [L, hk, D] in 64 bits, the first query at
    position p0.  Returns (out, lse, bound on |kernel - out|, bound on its lse)."""
    n, hq, D = q.shape
    L, hk = k.shape[0], k.shape[1]
    g = hq // hk
    q, k, v = q.double(), k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    pos = p0 + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(L, device=q.device)[None, :]
    see = (j >= 0) & (j < L) & (pos >= -(1 << 60))
    if causal:
        see = see & (j <= pos)
    if window:
        see = see & (pos - j < window)
    out = torch.zeros(n, hq, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    lse_bound = torch.zeros_like(lse)
    if L == 0:
        return out, lse, bound, lse_bound
    s = torch.einsum("nhd,lhd->hnl", q, k) * scale
    # |error of a score|: D products summed in f32, and the scaling
    ds = torch.einsum("nhd,lhd->hnl", q.abs(), k.abs()) * abs(scale) * (D + 4) * F32
    s = s.masked_fill(~see, -math.inf)
    some = see.any(1)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(s - top)
    tot = e.sum(-1, keepdim=True)
    w = e / torch.where(tot > 0, tot, torch.ones_like(tot))
    o = torch.einsum("hnl,lhd->nhd", w, v)
    mag = torch.einsum("hnl,lhd->nhd", w, v.abs())
    dmax = torch.where(see, ds, torch.zeros_like(ds)).amax(-1).transpose(0, 1)      # [n, hq]
    # scores' errors move each weight by a factor e^ds, twice (weights and their sum); the
    # f32 exponential and sums add 2^-18; a weight and the result are rounded to bf16 once
    out[:] = o
    bound[:] = U * o.abs() + (U + 2.5 * dmax[..., None] + 2.0 ** -18) * mag
    lse[some] = (top + torch.log(tot.clamp_min(1e-300))).squeeze(-1).transpose(0, 1)[some]
    lse_bound[:] = dmax + 2.0 ** -18 + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -20
    return out, lse, bound, lse_bound


class Paged:
    """A batch of sequences in a paged cache whose unused rows hold garbage: NaN in K, V and
    the scales.  lengths: (new tokens, cached positions) of each sequence."""

    def __init__(self, lib, lengths, hq, hk, D, page, fmt, seed=0, strided=False, spread=2.0, extra_pages=3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.lengths, self.hq, self.hk, self.D = lengths, hq, hk, D
        most = max(1, max(-(-kv // page) for _, kv in lengths))
        n_pages = len(lengths) * most + extra_pages
        self.cache = lib.kv_cache(n_pages, page, hk, D, fmt, device=DEV)
        for n in ("k", "v"):
            t = getattr(self.cache, n)
            if fmt == "bf16":
                t.fill_(math.nan)
            else:
                t.view(torch.uint8).fill_(0x7F)
                getattr(self.cache, n + "_scale").fill_(math.nan)
        order = torch.randperm(n_pages, generator=g, device=DEV)
        self.table = order[:len(lengths) * most].reshape(len(lengths), most).to(torch.int32).contiguous()
        slots, ks, vs = [], [], []
        for b, (_, kv) in enumerate(lengths):
            i = torch.arange(kv, device=DEV)
            slots.append(self.table[b].long()[i // page] * page + i % page)
            ks.append(rnd(kv, hk, D).to(torch.bfloat16))
            vs.append(rnd(kv, hk, D).to(torch.bfloat16))
        if sum(kv for _, kv in lengths):
            lib.kv_append(self.cache, torch.cat(ks), torch.cat(vs), torch.cat(slots).to(torch.int64))
        tokens = sum(n for n, _ in lengths)
        if strided:       # q a slice of a packed [tokens, (hq + 2 hk) D] buffer
            buf = (rnd(max(tokens, 1), (hq + 2 * hk) * D) * spread).to(torch.bfloat16)
            self.q = buf[:tokens, :hq * D].unflatten(1, (hq, D))
        else:
            self.q = (rnd(tokens, hq, D) * spread).to(torch.bfloat16)
        cu = [0]
        for n, _ in lengths:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=DEV)
        self.kv_len = torch.tensor([kv for _, kv in lengths], dtype=torch.int32, device=DEV)
        self.batch = lib.paged_batch(self.table, self.kv_len, self.cu_q)

    def rows64(self, b, n):
        """K or V of sequence b, [kv, hk, D] in 64 bits (what the cache stands for)."""
        kv = self.lengths[b][1]
        x = cache_values64(self.cache, n)[self.table[b].long()]
        return x.transpose(1, 2).flatten(0, 1)[:kv]

    def check(self, out, lse=None, scale=None, causal=True, window=0):
        scale = self.D ** -0.5 if scale is None else scale
        for b, (n, kv) in enumerate(self.lengths):
            r = slice(self.cu[b], self.cu[b] + n)
            if n == 0:
                continue
            ref, rl, bo, bl = attention64(self.q[r], self.rows64(b, "k"), self.rows64(b, "v"), kv - n, scale, causal,
                                          window)
            err = (out[r].double() - ref).abs()
            assert bool(torch.isfinite(out[r].double()).all()), f"sequence {b}: not finite"
            over = float((err - 1.01 * bo).max())
            assert over <= 0, f"sequence {b} ({n} of {kv}): {over:.3e} over the bound (error {float(err.max()):.3e})"
            if lse is not None:
                none = torch.isneginf(rl)
                assert torch.equal(torch.isneginf(lse[r]), none)
                d = (lse[r].double() - rl).abs()[~none]
                assert bool((d <= bl[~none]).all()), f"sequence {b}: lse off by {float(d.max()):.3e}"
