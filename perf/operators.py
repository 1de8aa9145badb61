"""Measured cases of the serving operators between the Q/K/V and the output projection:
rotary positions, the paged K/V cache (written with quantisation, read back) and the
attention of new tokens over that cache.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, with ``own`` set, by the library's entry points.  ``exact``
gives the same results from the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
TINY = 1.17549435e-38                     # smallest normal f32: the least scale of a cached row
TOP = {"int8": 127.0, "fp8": 448.0}       # largest code of a format
STORE = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases

def _rotary(name, tokens, hq, hk, dim, rot, layout, inverse, packed):
    return {"name": name, "op": "rotary", "tokens": tokens, "hq": hq, "hk": hk, "dim": dim, "rot": rot,
            "layout": layout, "inverse": inverse, "packed": packed}


def _append(name, tokens, hq, hk, dim, rot, layout, fmt, page):
    return {"name": name, "op": "append", "tokens": tokens, "hq": hq, "hk": hk, "dim": dim, "rot": rot,
            "layout": layout, "fmt": fmt, "page": page}


def _read(name, batch, kv_lo, kv_hi, hk, dim, fmt, page):
    return {"name": name, "op": "read", "batch": batch, "kv_lo": kv_lo, "kv_hi": kv_hi, "hk": hk, "dim": dim,
            "fmt": fmt, "page": page}


def _attn(name, batch, new_lo, new_hi, kv_lo, kv_hi, hq, hk, dim, fmt, page, window=0):
    return {"name": name, "op": "attn", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "kv_lo": kv_lo,
            "kv_hi": kv_hi, "hq": hq, "hk": hk, "dim": dim, "fmt": fmt, "page": page, "window": window}


def listed():
    return [
        # one decode step of a small block (14:2 heads of 64): latency of a single launch
        _rotary("rotary_decode_16", 16, 14, 2, 64, 64, "half", False, False),
        # a prefill of 8192 tokens, 32:8 heads of 128, neighbouring features paired
        _rotary("rotary_prefill_8192", 8192, 32, 8, 128, 128, "interleaved", False, False),
        # the gradient of an odd number of tokens, a quarter of wide heads rotated, q and k
        # slices of one packed q/k/v buffer
        _rotary("rotary_grad_4099", 4099, 16, 16, 256, 64, "half", True, True),
        # the cache write of one decode step of 64 sequences, q and k rotated on the way
        _append("append_decode_64", 64, 32, 8, 128, 128, "half", "int8", 16),
        # the cache write of a whole prefill
        _append("append_prefill_8192", 8192, 32, 8, 128, 128, "half", "fp8", 64),
        # eight sequences' K and V out of the cache (to move them, or to train on them)
        _read("read_back_8", 8, 100, 6001, 8, 128, "int8", 32),
        # one sequence, one token, a short cache: latency
        _attn("attn_decode_1", 1, 1, 1, 777, 777, 14, 2, 64, "bf16", 16),
        # a decode step of 64 sequences of very different lengths
        _attn("attn_decode_64_int8", 64, 1, 1, 200, 8192, 32, 8, 128, "int8", 64),
        # a decode step of few sequences with long caches
        _attn("attn_decode_4_long", 4, 1, 1, 50001, 65536, 32, 8, 128, "bf16", 64),
        # prefill chunks over a long, already filled cache
        _attn("attn_chunk_512_fp8", 2, 512, 512, 15873, 16384, 32, 8, 128, "fp8", 64),
        # the first prefill of four sequences of 2048 tokens: causal, compute-bound
        _attn("attn_prefill_4x2048", 4, 2048, 2048, 2048, 2048, 32, 8, 128, "bf16", 128),
        # decode and prefill mixed in one batch, wide heads without sharing, a window
        _attn("attn_mixed_24", 24, 1, 257, 300, 4096, 16, 16, 256, "bf16", 32, 1024),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "read", "attn", "attn", "attn"])
    hq, hk, dim = rng.choice([(14, 2, 64), (32, 8, 128), (16, 16, 256), (8, 1, 128), (12, 4, 64), (28, 4, 128),
                              (16, 8, 256)])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["bf16", "int8", "fp8"])
    layout = rng.choice(["half", "interleaved"])
    rot = rng.choice([dim, dim // 2, dim // 4])
    if op == "rotary":
        c = _rotary("", _spread(rng, 1, 8192), hq, hk, dim, rot, layout, rng.random() < 0.5, rng.random() < 0.5)
    elif op == "append":
        c = _append("", _spread(rng, 1, 8192), hq, hk, dim, rot, layout, fmt, page)
    elif op == "read":
        hi = _spread(rng, 30, 4001)
        c = _read("", _spread(rng, 1, 8), max(1, hi // rng.randint(1, 8)), hi, hk, dim, fmt, page)
    else:
        kind = rng.choice(["decode", "chunk", "prefill", "mixed"])
        window = rng.choice([0, 0, 0, 333, 1024])
        most = 9e8 / (2 * hk * (2 * dim if fmt == "bf16" else dim + 4))     # cached keys of a call at most
        if kind == "decode":
            batch = _spread(rng, 1, 64)
            hi = _spread(rng, 100, min(65536, int(most / batch)))
            c = _attn("", batch, 1, 1, max(1, hi // rng.randint(1, 8)), hi, hq, hk, dim, fmt, page, window)
        elif kind == "chunk":
            new = _spread(rng, 2, 512)
            hi = _spread(rng, 600, 8192)
            c = _attn("", rng.randint(1, 2), new, new, max(new, hi - rng.randint(0, 500)), hi, hq, hk, dim, fmt,
                      page, window)
        elif kind == "prefill":
            hi = _spread(rng, 17, 2048)
            c = _attn("", rng.randint(1, 4), hi, hi, hi, hi, hq, hk, dim, fmt, page, window)
        else:
            hi = _spread(rng, 260, 4096)
            batch = rng.randint(2, min(24, int(most / hi)))
            c = _attn("", batch, 1, _spread(rng, 2, 257), max(257, hi // 4), hi, hq, hk, dim, fmt, page, window)
    del c["name"]
    return c


def _lengths(n, lo, hi, stride):
    """n whole numbers spread evenly over [lo, hi], in a mixed order (the same every time)."""
    even = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]
    step = next(s for s in range(stride, stride + 2 * n + 2) if math.gcd(s, n) == 1)
    return [even[i * step % n] for i in range(n)]


def _batch(case):
    """(new tokens, cached keys) of each sequence of an attention case."""
    kv = _lengths(case["batch"], case["kv_lo"], case["kv_hi"], 7)
    new = _lengths(case["batch"], case["new_lo"], case["new_hi"], 5)
    return [min(a, b) for a, b in zip(new, kv)], kv


def _visible(new, kv, window):
    """Visible (query, key) pairs of one sequence, and its keys that any query sees."""
    first = kv - new + 1
    if window == 0:
        return sum(range(first, kv + 1)), kv
    seen = kv - max(0, first - window)
    return sum(min(p, window) for p in range(first, kv + 1)), seen


def work(case):
    c = case
    if c["op"] == "rotary":
        feats = c["tokens"] * (c["hq"] + c["hk"]) * c["dim"]
        turned = c["tokens"] * (c["hq"] + c["hk"]) * c["rot"]
        return {"bytes": 4.0 * feats + c["tokens"] * (4.0 * c["rot"] + 4), "flops": 3.0 * turned}
    size = 2 if c["fmt"] == "bf16" else 1
    row = c["dim"] * size + (0 if c["fmt"] == "bf16" else 4)       # one cached row of K or V
    if c["op"] == "append":
        t = c["tokens"]
        return {"bytes": t * (4.0 * c["hq"] * c["dim"] + 4.0 * c["hk"] * c["dim"] + 2.0 * c["hk"] * row
                              + 4.0 * c["rot"] + 12),
                "flops": t * (3.0 * (c["hq"] + c["hk"]) * c["rot"] + 4.0 * c["hk"] * c["dim"])}
    if c["op"] == "read":
        rows = 2.0 * c["hk"] * sum(_lengths(c["batch"], c["kv_lo"], c["kv_hi"], 7))
        return {"bytes": rows * (row + 2 * c["dim"]), "flops": rows * c["dim"]}
    seen = [_visible(n, l, c["window"]) for n, l in zip(*_batch(c))]
    tokens = sum(_batch(c)[0])
    return {"bytes": 4.0 * tokens * c["hq"] * c["dim"] + 2.0 * c["hk"] * row * sum(s[1] for s in seen),
            "flops": 4.0 * c["hq"] * c["dim"] * sum(s[0] for s in seen)}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(torch.bfloat16)


def _tables(positions, rot, base=10000.0):
    """cos, sin [positions, rot/2] of p * base^(-2c/rot), rounded once to f32."""
    w = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * w
    return a.cos().float(), a.sin().float()


def _rope(case, g):
    n_pos = max(case["tokens"], 4096)
    cos, sin = _tables(n_pos, case["rot"])
    pos = torch.randint(0, n_pos, (case["tokens"],), generator=g, device=DEV, dtype=torch.int32)
    return {"cos": cos, "sin": sin, "pos": pos, "layout": case["layout"]}


def _quantise(x, fmt):
    """(codes, scales) of rows x [..., D] in f32."""
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.clamp(amax * (1.0 / TOP[fmt]), min=TINY)
    fine = torch.isfinite(amax)
    scale = torch.where(fine, scale, float("nan"))
    y = torch.where(fine, x * torch.reciprocal(scale), 0.0).clamp(-TOP[fmt], TOP[fmt])
    y = y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return y, scale.squeeze(-1)


def _pages(g, fmt, n_pages, hk, page, dim):
    """A filled cache's tensors: k, v [n_pages, hk, page, dim] and their scales."""
    out = {}
    for n in ("k", "v"):
        x = _normal(g, n_pages, hk, page, dim)
        if fmt == "bf16":
            out[n], out[n + "_scale"] = x, None
        else:
            out[n], out[n + "_scale"] = _quantise(x.float(), fmt)
        del x
    return out


def _page_table(g, lengths, page):
    """A random assignment of pages to sequences, and the number of pages of the pool."""
    most = max(-(-n // page) for n in lengths)
    used = len(lengths) * most
    pool = used + 8
    order = torch.randperm(pool, generator=g, device=DEV)[:used]
    return order.to(torch.int32).reshape(len(lengths), most), pool


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    s = {"case": c}
    if c["op"] == "rotary":
        t, dim, hq, hk = c["tokens"], c["dim"], c["hq"], c["hk"]
        if c["packed"]:
            both = _normal(g, t, (hq + 2 * hk) * dim)
            s["q"] = both[:, :hq * dim].unflatten(1, (hq, dim))
            s["k"] = both[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
        else:
            s["q"], s["k"] = _normal(g, t, hq, dim), _normal(g, t, hk, dim)
        s["rope"] = _rope(c, g)
        return s
    if c["op"] == "append":
        t, dim, hq, hk, page = c["tokens"], c["dim"], c["hq"], c["hk"], c["page"]
        # k and v as the projections give them; slots of a pool twice as large as the call
        s["q"], s["k"], s["v"] = _normal(g, t, hq, dim), _normal(g, t, hk, dim), _normal(g, t, hk, dim)
        s["rope"] = _rope(c, g)
        n_pages = -(-2 * t // page) + 1
        s["slots"] = torch.randperm(n_pages * page, generator=g, device=DEV)[:t].to(torch.int64)
        s["pages"] = _pages(g, c["fmt"], n_pages, hk, page, dim)
    elif c["op"] == "read":
        lengths = _lengths(c["batch"], c["kv_lo"], c["kv_hi"], 7)
        s["table"], n_pages = _page_table(g, lengths, c["page"])
        s["total"] = sum(lengths)
        s["cu_kv"] = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=DEV)
        s["pages"] = _pages(g, c["fmt"], n_pages, c["hk"], c["page"], c["dim"])
    else:
        new, kv = _batch(c)
        s["table"], n_pages = _page_table(g, kv, c["page"])
        s["tokens"], s["most_new"], s["most_kv"] = sum(new), max(new), max(kv)
        s["cu_q"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
        # scores with a spread of about two: some keys matter, none alone
        s["q"] = _normal(g, s["tokens"], c["hq"], c["dim"], scale=2.0)
        s["pages"] = _pages(g, c["fmt"], n_pages, c["hk"], c["page"], c["dim"])
    if own:
        # the handles a serving program keeps: the cache over the same tensors, and the
        # batch's description, which all layers of a step share
        from rank_mlp_gb300 import binding as lora
        s["cache"] = lora.KVCache(s["pages"]["k"], s["pages"]["v"], s["pages"]["k_scale"], s["pages"]["v_scale"])
        if c["op"] == "attn":
            s["batch"] = lora.paged_batch(s["table"], s["kv_len"], s["cu_q"])
    return s


# ------------------------------------------------------------------ plain forms

def _turn(x, rope, inverse=False):
    """x [T, heads, D] rotated in f32 (not rounded)."""
    x = x.float()
    half = rope["cos"].shape[1]
    cos = rope["cos"][rope["pos"].long()][:, None, :]
    sin = rope["sin"][rope["pos"].long()][:, None, :]
    if inverse:
        sin = -sin
    if rope["layout"] == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _values(pages, n):
    """The f32 values of a cache's k or v pages."""
    x = pages[n].float()
    return x if pages[n + "_scale"] is None else x * pages[n + "_scale"][..., None]


def _plain_append(s):
    page = s["pages"]["k"].shape[2]
    at, off = s["slots"] // page, s["slots"] % page
    for n, x in (("k", _turn(s["k"], s["rope"])), ("v", s["v"].float())):
        dst, scale = s["pages"][n], s["pages"][n + "_scale"]
        if scale is None:
            dst[at, :, off] = x.to(torch.bfloat16)
        else:
            code, sc = _quantise(x, s["case"]["fmt"])
            dst.view(torch.uint8)[at, :, off] = code.view(torch.uint8)
            scale[at, :, off] = sc
    return {"q": _turn(s["q"], s["rope"]).to(torch.bfloat16), **{n: t for n, t in s["pages"].items() if t is not None}}


def _plain_read(s):
    cu, page = s["cu_kv"].long(), s["pages"]["k"].shape[2]
    row = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[seq]
    at, off = s["table"].long()[seq, i // page], i % page
    out = {}
    for n in ("k", "v"):
        x = s["pages"][n].view(torch.uint8 if s["case"]["fmt"] != "bf16" else torch.bfloat16)[at, :, off]
        x = x.view(s["pages"][n].dtype).float()
        if s["pages"][n + "_scale"] is not None:
            x = x * s["pages"][n + "_scale"][at, :, off][..., None]
        out[n] = x.to(torch.bfloat16)
    return out


def _plain_attn(s):
    c = s["case"]
    hq, hk, dim, page = c["hq"], c["hk"], c["dim"], c["page"]
    group, batch, most, keys = hq // hk, c["batch"], s["most_new"], s["most_kv"]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    new = cu[1:] - cu[:-1]
    # K and V of every sequence side by side: [batch, hk, keys, dim], zero past its length
    j = torch.arange(keys, device=DEV)
    alive = j[None, :] < kv[:, None]

    def gather(n):
        x = s["pages"][n][s["table"].long()] if c["fmt"] == "bf16" else \
            s["pages"][n].view(torch.uint8)[s["table"].long()].view(s["pages"][n].dtype)
        x = x.float()
        if s["pages"][n + "_scale"] is not None:
            x = x * s["pages"][n + "_scale"][s["table"].long()][..., None]
        x = x.permute(0, 2, 1, 3, 4).reshape(batch, hk, -1, dim)[:, :, :keys]
        return torch.where(alive[:, None, :, None], x, 0.0)

    # queries side by side: [batch, hk, most * group, dim]
    i = torch.arange(most, device=DEV)
    src = (cu[:-1, None] + i[None, :]).clamp(max=s["tokens"] - 1)
    q = s["q"][src].float().reshape(batch, most, hk, group, dim).permute(0, 2, 1, 3, 4)
    score = torch.matmul(q.reshape(batch, hk, most * group, dim), gather("k").transpose(2, 3)) / math.sqrt(dim)
    p = kv[:, None] - new[:, None] + i[None, :]                      # positions [batch, most]
    see = alive[:, None, :] & (j[None, None, :] <= p[:, :, None])
    if c["window"]:
        see = see & (p[:, :, None] - j[None, None, :] < c["window"])
    see = see[:, None, :, None, :].expand(batch, 1, most, group, keys).reshape(batch, 1, most * group, keys)
    score = torch.where(see, score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, gather("v")) / torch.where(total > 0, total, 1.0)
    o = o.reshape(batch, hk, most, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, most, hq, dim)
    row = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    return o[seq, row - cu[seq]].to(torch.bfloat16)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "rotary":
            inv = s["case"]["inverse"]
            return [_turn(s["q"], s["rope"], inv).to(torch.bfloat16), _turn(s["k"], s["rope"], inv).to(torch.bfloat16)]
        return {"append": _plain_append, "read": _plain_read, "attn": _plain_attn}[op](s)
    from rank_mlp_gb300 import binding as lora
    if op == "rotary":
        return list(lora.rotary(s["q"], s["k"], rope=s["rope"], inverse=s["case"]["inverse"]))
    if op == "append":
        q = lora.kv_append(s["cache"], s["k"], s["v"], s["slots"], q=s["q"], rope=s["rope"])
        return {"q": q, **{n: t for n, t in s["pages"].items() if t is not None}}
    if op == "read":
        k, v = lora.kv_read(s["cache"], s["table"], s["cu_kv"], s["total"])
        return {"k": k, "v": v}
    return lora.paged_attention(s["q"], s["cache"], s["batch"], window=s["case"]["window"])


# ------------------------------------------------------------------ the definitions in 64 bits

def _turn64(x, rope, inverse):
    """Rotation as a complex product, in 64 bits."""
    h = rope["cos"].shape[1]
    sign = -1.0 if inverse else 1.0
    w = torch.complex(rope["cos"].double(), sign * rope["sin"].double())[rope["pos"].long()].unsqueeze(1)
    y = x.double().clone()
    first = slice(0, h) if rope["layout"] == "half" else slice(0, 2 * h, 2)
    second = slice(h, 2 * h) if rope["layout"] == "half" else slice(1, 2 * h, 2)
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _sequence64(pages, n, table, length):
    """Rows [0, length) of one sequence's K or V: [length, hk, dim] in 64 bits."""
    t = table.long()
    x = pages[n].view(torch.uint8 if pages[n].element_size() == 1 else torch.int16)[t].view(pages[n].dtype).double()
    if pages[n + "_scale"] is not None:
        x = x * pages[n + "_scale"][t].double().unsqueeze(-1)
    return x.transpose(1, 2).flatten(0, 1)[:length]


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rotary":
        return [_turn64(s[n], s["rope"], c["inverse"]) for n in ("q", "k")]
    if c["op"] == "append":
        out = {"q": _turn64(s["q"], s["rope"], False)}
        for n, x in (("k", _turn64(s["k"], s["rope"], False)), ("v", s["v"].double())):
            old, scales, page = s["pages"][n], s["pages"][n + "_scale"], c["page"]
            flat = old.double().transpose(1, 2).flatten(0, 1).clone()          # [slots, hk, dim]
            if scales is None:
                flat[s["slots"]] = x
            else:
                sc = scales.double().transpose(1, 2).flatten(0, 1).clone()
                amax = x.abs().max(-1).values
                sc[s["slots"]] = amax / TOP[c["fmt"]]
                flat[s["slots"]] = x / (amax / TOP[c["fmt"]]).unsqueeze(-1)
                out[n + "_scale"] = sc.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
            # int8 codes are whole numbers: held to equality, without a 64-bit value
            out[n] = None if c["fmt"] == "int8" else flat.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
        return out
    if c["op"] == "read":
        lengths = _lengths(c["batch"], c["kv_lo"], c["kv_hi"], 7)
        return {n: torch.cat([_sequence64(s["pages"], n, s["table"][b], lengths[b]) for b in range(c["batch"])])
                for n in ("k", "v")}
    new, kv = _batch(c)
    group, out, at = c["hq"] // c["hk"], [], 0
    if 4.0 * c["hq"] * c["dim"] * sum(a * b for a, b in zip(new, kv)) > 4e12:
        return None
    for b in range(c["batch"]):
        k, v = (_sequence64(s["pages"], n, s["table"][b], kv[b]).transpose(0, 1) for n in ("k", "v"))
        q = s["q"][at:at + new[b]].double()
        at += new[b]
        p = torch.arange(kv[b] - new[b], kv[b], device=DEV)[:, None]
        j = torch.arange(kv[b], device=DEV)[None, :]
        hidden = (j > p) | ((p - j >= c["window"]) if c["window"] else torch.zeros_like(j > p))
        heads = []
        for h in range(c["hq"]):
            z = (q[:, h] @ k[h // group].T) * c["dim"] ** -0.5
            heads.append(torch.softmax(z.masked_fill(hidden, float("-inf")), -1) @ v[h // group])
        out.append(torch.stack(heads, 1))
    return torch.cat(out)
