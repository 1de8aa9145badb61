"""Measured cases of the operators that a training step runs around the block's projections:
the RMS norm with the residual's addition (and its gradient), the cross entropy of a frozen
head with its gradient, clipping by the global gradient norm, and the clipped sum of
per-example gradients.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, with ``own`` set, by the library's entry points.  ``exact``
gives the same results from the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
TINY = 1.17549435e-38                     # smallest normal f32: the least scale of a row
TOP = 448.0                               # largest e4m3 value
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _norm(name, tokens, heads, h, residual, fmt, packed=False, offset=0.0):
    return {"name": name, "op": "norm", "tokens": tokens, "heads": heads, "h": h, "residual": residual, "fmt": fmt,
            "packed": packed, "offset": offset}


def _norm_grad(name, tokens, heads, h, residual, dweight, offset=0.0):
    return {"name": name, "op": "norm_grad", "tokens": tokens, "heads": heads, "h": h, "residual": residual,
            "dweight": dweight, "offset": offset}


def _ce(name, tokens, h, vocab, grad, reduction="mean", scale=1.0, softcap=0.0, smoothing=0.0, ignored=0.1):
    return {"name": name, "op": "ce", "tokens": tokens, "h": h, "vocab": vocab, "grad": grad, "reduction": reduction,
            "scale": scale, "softcap": softcap, "smoothing": smoothing, "ignored": ignored}


def _clip(name, layers, h, inter, kv, rank, dtype, odd=0, norm="2"):
    return {"name": name, "op": "clip", "layers": layers, "h": h, "inter": inter, "kv": kv, "rank": rank, "dtype": dtype,
            "odd": odd, "norm": norm}


def _examples(name, n, h, inter, rank, layers, known):
    return {"name": name, "op": "examples", "n": n, "h": h, "inter": inter, "rank": rank, "layers": layers,
            "known": known}


def listed():
    return [
        # one step of a few tokens of a small block: the latency of a launch
        _norm("norm_16", 16, 1, 896, True, "bf16"),
        # the residual stream of a long batch, for a projection that takes 8-bit rows
        _norm("norm_8192_fp8", 8192, 1, 4096, True, "fp8"),
        # the norm of each query head, a slice of one packed q/k/v buffer
        _norm("norm_heads_4099", 4099, 32, 128, False, "bf16", packed=True),
        # its gradient in a training step, with the residual stream's and the weight's
        _norm_grad("norm_grad_4095", 4095, 1, 4096, True, True),
        # the loss of a short example on a small model: both passes read the whole head
        _ce("ce_64", 64, 896, 32000, True),
        # a training step of a small model: the vocabulary outweighs the block
        _ce("ce_4095", 4095, 896, 131072, True),
        # evaluation: the loss alone, smoothed, over a vocabulary of odd size
        _ce("ce_eval_2048", 2048, 4096, 50257, False, smoothing=0.1),
        # a training step with capped logits
        _ce("ce_4096_softcap", 4096, 4096, 131072, True, "sum", softcap=30.0),
        # the adapters of a whole model: hundreds of tensors of two shapes
        _clip("clip_adapters_448", 32, 4096, 14336, 1024, 16, "bf16"),
        # gradients accumulated in 32 bits, tensors of odd sizes
        _clip("clip_f32_odd", 24, 4096, 14336, 1024, 64, "f32", odd=3),
        # DP-SGD on a tiny block: latency
        _examples("examples_8_tiny", 8, 128, 344, 8, 1, False),
        # DP-SGD, 32 examples' gradients of two blocks' MLPs
        _examples("examples_32", 32, 4096, 14336, 16, 2, False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "ce", "ce", "clip", "examples"])
    offset = rng.choice([0.0, 0.0, 1.0])
    if op in ("norm", "norm_grad"):
        if rng.random() < 0.3:
            heads, h = rng.choice([(14, 64), (32, 128), (8, 128), (16, 256)])
            tokens = _spread(rng, 1, 8192)
        else:
            heads, h = 1, 8 * _spread(rng, 16, 1024)
            tokens = _spread(rng, 1, min(8192, (1 << 25) // h))
        if op == "norm":
            c = _norm("", tokens, heads, h, heads == 1 and rng.random() < 0.7, rng.choice(["bf16", "fp8"]),
                      rng.random() < 0.4, offset)
        else:
            c = _norm_grad("", tokens, heads, h, heads == 1 and rng.random() < 0.7, rng.random() < 0.5, offset)
    elif op == "ce":
        h = 8 * _spread(rng, 16, 512)
        vocab = _spread(rng, 500, 131072)
        tokens = _spread(rng, 1, min(8192, int(2e12 / (h * vocab))))
        c = _ce("", tokens, h, vocab, rng.random() < 0.75, rng.choice(["mean", "sum"]), rng.choice([1.0, 1.0, 0.25]),
                rng.choice([0.0, 0.0, 30.0, 15.0]), rng.choice([0.0, 0.0, 0.1]), rng.choice([0.0, 0.1, 0.6]))
    elif op == "clip":
        h = 8 * _spread(rng, 16, 512)
        c = _clip("", rng.randint(1, 32), h, 8 * (h * 3 // 8), max(8, h // 4), rng.choice([4, 8, 16, 32]),
                  rng.choice(["bf16", "f32"]), rng.choice([0, 0, 1, 5]), rng.choice(["2", "2", "inf"]))
    else:
        h = 8 * _spread(rng, 16, 512)
        c = _examples("", _spread(rng, 1, 32), h, 8 * (h * 3 // 8), rng.choice([4, 8, 16]), rng.randint(1, 2),
                      rng.random() < 0.4)
    del c["name"]
    return c


def _adapter_sizes(c):
    """Elements of the adapters' gradients of a model, A and B of each projection."""
    r, h, i, kv = c["rank"], c["h"], c["inter"], c["kv"]
    one = []
    for a, b in ((h, h), (h, kv), (h, kv), (h, h), (h, i), (h, i), (i, h)):
        one += [r * a + c["odd"], r * b + c["odd"]]
    return one * c["layers"]


def _example_sizes(c):
    """Elements of one example's adapter gradients of the MLPs."""
    r, h, i = c["rank"], c["h"], c["inter"]
    return [r * h, i * r, r * h, i * r, r * i, h * r] * c["layers"]


def work(case):
    c = case
    if c["op"] == "norm":
        rows, h = c["tokens"] * c["heads"], c["h"]
        per = 2 * h + (4 * h if c["residual"] else 0) + (2 * h if c["fmt"] == "bf16" else h + 4) + 4
        return {"bytes": float(rows * per + 2 * h), "flops": 5.0 * rows * h}
    if c["op"] == "norm_grad":
        rows, h = c["tokens"] * c["heads"], c["h"]
        per = 6 * h + (2 * h if c["residual"] else 0) + 4
        return {"bytes": float(rows * per + 2 * h + (2 * h if c["dweight"] else 0)), "flops": 9.0 * rows * h}
    if c["op"] == "ce":
        m, h, v = c["tokens"], c["h"], c["vocab"]
        seen = m - int(m * c["ignored"])
        return {"bytes": 2.0 * v * h + m * (2.0 * h + 16) + (2.0 * m * h if c["grad"] else 0.0),
                "flops": (4.0 if c["grad"] else 2.0) * seen * h * v}
    if c["op"] == "clip":
        n = sum(_adapter_sizes(c))
        return {"bytes": 2.0 * n * (2 if c["dtype"] == "bf16" else 4), "flops": 3.0 * n}
    n = sum(_example_sizes(c))
    return {"bytes": 2.0 * c["n"] * n + 4.0 * n, "flops": (2.0 if c["known"] else 4.0) * c["n"] * n}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _shape(c):
    return (c["tokens"], c["heads"], c["h"]) if c["heads"] > 1 else (c["tokens"], c["h"])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    s = {"case": c}
    if c["op"] in ("norm", "norm_grad"):
        # rows of unlike size, as a residual stream has them; weights around one (or zero)
        h = c["h"]
        s["weight"] = (1.0 - c["offset"] + 0.2 * torch.randn(h, generator=g, device=DEV)).to(torch.bfloat16)
        size = torch.exp(torch.randn(c["tokens"], generator=g, device=DEV))
        if c["heads"] > 1:
            size = size[:, None]
        shape = _shape(c)
        rows = lambda: (torch.randn(*shape, generator=g, device=DEV) * size[..., None]).to(torch.bfloat16)  # noqa: E731
        s["x"] = rows()
        if c.get("packed"):
            wide = _normal(g, c["tokens"], 2 * c["heads"] * h)
            x = wide[:, :c["heads"] * h]
            x = x.unflatten(1, (c["heads"], h)) if c["heads"] > 1 else x
            s["x"] = x.copy_(s["x"])
        if c["op"] == "norm":
            s["residual"] = rows() if c["residual"] else None
        else:
            s["ds"] = _normal(g, *shape) if c["residual"] else None
            s["dy"] = _normal(g, *shape)
            ms = s["x"].double().square().mean(-1)
            s["rstd"] = torch.rsqrt(ms + EPS).float()
    elif c["op"] == "ce":
        m, h, v = c["tokens"], c["h"], c["vocab"]
        s["W"] = _normal(g, v, h, scale=h ** -0.5)
        s["labels"] = torch.randint(0, v, (m,), generator=g, device=DEV)
        # logits with a spread of about two, the label's raised by up to sixteen: from
        # tokens the model does not expect to ones it is sure of
        lift = torch.rand(m, 1, generator=g, device=DEV) * 16.0
        s["x"] = (2.0 * torch.randn(m, h, generator=g, device=DEV) + lift * s["W"][s["labels"]].float()).to(torch.bfloat16)
        hide = torch.randperm(m, generator=g, device=DEV)[:int(m * c["ignored"])]
        s["labels"][hide] = -100
    elif c["op"] == "clip":
        # the gradients lie one after the other in one buffer, as reducing them leaves them;
        # the result goes to another (a pass does not change what the next one reads)
        sizes = _adapter_sizes(c)
        dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["flat"] = _normal(g, sum(sizes), scale=1e-2, dtype=dtype)
        s["clipped"] = torch.empty_like(s["flat"])
        s["max_norm"] = 1.0 if c["norm"] == "2" else 0.01
    else:
        sizes = _example_sizes(c)
        size = torch.exp(torch.randn(c["n"], 1, generator=g, device=DEV))
        s["grads"] = [(torch.randn(c["n"], k, generator=g, device=DEV) * size * 1e-3).to(torch.bfloat16) for k in sizes]
        s["max_norm"] = 1e-3 * math.sqrt(sum(sizes))
        s["known"] = sum(t.double().square().sum(1) for t in s["grads"]).float() if c["known"] else None
    if own:
        # the lists of tensors that a program keeps from step to step
        from rank_mlp_gb300 import binding as lora
        if c["op"] == "clip":
            s["list"] = lora.tensor_list(list(s["flat"].split(sizes)))
            s["out"] = lora.tensor_list(list(s["clipped"].split(sizes)))
        elif c["op"] == "examples":
            s["list"] = lora.tensor_list(s["grads"])
    return s


# ------------------------------------------------------------------ plain forms

def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    out = {}
    if s["residual"] is not None:
        out["s"] = (x + s["residual"].float()).to(torch.bfloat16)
        x = out["s"].float()
    out["rstd"] = torch.rsqrt(x.square().mean(-1) + EPS)
    y = x * out["rstd"][..., None] * (s["weight"].float() + c["offset"])
    if c["fmt"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    else:
        scale = torch.clamp(y.abs().amax(-1) * (1.0 / TOP), min=TINY)
        out["y"] = (y * torch.reciprocal(scale)[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
        out["scale"] = scale
    return out


def _plain_norm_grad(s):
    c = s["case"]
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][..., None]
    g = dy * (s["weight"].float() + c["offset"])
    n = x * rstd
    dx = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    out = {"dx": dx.to(torch.bfloat16)}
    if c["dweight"]:
        out["dweight"] = (dy * n).flatten(0, -2).sum(0).to(torch.bfloat16)
    return out


def _plain_ce(s):
    c = s["case"]
    x, w, y = s["x"].float(), s["W"].float(), s["labels"]
    seen = y != -100
    at = torch.where(seen, y, 0)[:, None]
    z = torch.matmul(x, w.T)
    z.mul_(c["scale"])
    if c["softcap"]:
        z.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    top = z.amax(1, keepdim=True)
    lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
    eps, v = c["smoothing"], c["vocab"]
    loss = lse - (1.0 - eps) * z.gather(1, at)[:, 0]
    if eps:
        loss = loss - eps * z.mean(1)
    loss = torch.where(seen, loss, 0.0)
    count = seen.sum().clamp(min=1).float() if c["reduction"] == "mean" else torch.ones((), device=DEV)
    out = {"total": loss.sum() / count, "loss": loss, "lse": torch.where(seen, lse, 0.0)}
    if c["grad"]:
        slope = 1.0 - (z / c["softcap"]).square() if c["softcap"] else None
        dz = z.sub_(lse[:, None]).exp_()
        dz.scatter_add_(1, at, torch.full_like(at, -(1.0 - eps), dtype=torch.float32))
        if eps:
            dz.sub_(eps / v)
        if slope is not None:
            dz.mul_(slope)
        dz.mul_(torch.where(seen, c["scale"] / count, 0.0)[:, None])
        out["dx"] = torch.matmul(dz, w).to(torch.bfloat16)
    return out


def _plain_clip(s):
    g = s["flat"].float()
    norm = g.abs().amax() if s["case"]["norm"] == "inf" else g.square().sum().sqrt()
    s["clipped"].copy_(g * torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0))
    return {"norm": norm, "clipped": s["clipped"]}


def _plain_examples(s):
    wide = [t.float() for t in s["grads"]]
    sq = s["known"] if s["known"] is not None else torch.stack([t.square().sum(1) for t in wide]).sum(0)
    keep = torch.clamp(s["max_norm"] / sq.sqrt(), max=1.0) / s["case"]["n"]
    return {"sums": [(t * keep[:, None]).sum(0) for t in wide], "sq_norms": sq}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "ce": _plain_ce, "clip": _plain_clip,
                "examples": _plain_examples}[op](s)
    from rank_mlp_gb300 import binding as lora
    if op == "norm":
        y, total, rstd = lora.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, offset=c["offset"],
                                       format=c["fmt"], training=True)
        out = {"rstd": rstd}
        if s["residual"] is not None:
            out["s"] = total
        return out | ({"y": y} if c["fmt"] == "bf16" else {"y": y[0], "scale": y[1]})
    if op == "norm_grad":
        dx, dw = lora.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], offset=c["offset"], ds=s["ds"],
                                        dweight=c["dweight"])
        return {"dx": dx} | ({"dweight": dw} if c["dweight"] else {})
    if op == "ce":
        total, loss, lse, dx = lora.linear_cross_entropy(
            s["x"], s["W"], s["labels"], scale=c["scale"], softcap=c["softcap"], smoothing=c["smoothing"],
            reduction=c["reduction"], grad=c["grad"])
        return {"total": total, "loss": loss, "lse": lse} | ({"dx": dx} if c["grad"] else {})
    if op == "clip":
        norm = lora.clip_grad_norm(s["list"], s["max_norm"], norm_type=float(c["norm"]), out=s["out"])
        return {"norm": norm, "clipped": s["clipped"]}
    sums, sq = lora.clip_examples(s["list"], s["max_norm"], sq_norms=s["known"], scale=1.0 / c["n"])
    return {"sums": sums, "sq_norms": sq}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        x = s["x"].double()
        out = {}
        if s["residual"] is not None:
            # the stream is rounded where it is stored, and the norm is of what is stored
            x = x + s["residual"].double()
            out["s"] = x
            x = x.to(torch.bfloat16).double()
        power = torch.linalg.vector_norm(x, dim=-1) ** 2 / c["h"]
        out["rstd"] = (power + EPS) ** -0.5
        y = x / torch.sqrt(power + EPS).unsqueeze(-1) * (s["weight"].double() + c["offset"])
        if c["fmt"] == "fp8":
            out["scale"] = y.abs().max(-1).values / TOP
            y = y / out["scale"].unsqueeze(-1)
        out["y"] = y
        return out
    if c["op"] == "norm_grad":
        # from the derivative of each normalised feature: (1 - n n^T / h) g / rms
        x, dy = s["x"].double(), s["dy"].double()
        inv = s["rstd"].double().unsqueeze(-1)
        g = dy * (s["weight"].double() + c["offset"])
        along = (g * x).sum(-1, keepdim=True) / c["h"]
        dx = inv * g - inv ** 3 * along * x
        out = {"dx": dx if s["ds"] is None else dx + s["ds"].double()}
        if c["dweight"]:
            out["dweight"] = torch.einsum("rh,rh,r->h", dy.flatten(0, -2), x.flatten(0, -2), inv.flatten())
        return out
    if c["op"] == "ce":
        m, h, v = c["tokens"], c["h"], c["vocab"]
        if m * h * v > 3e12:
            return None
        w, eps, cap = s["W"].double(), c["smoothing"], c["softcap"]
        loss, lses, grads = [], [], []
        count = max(1, int((s["labels"] != -100).sum())) if c["reduction"] == "mean" else 1
        for a in range(0, m, 512):
            x, y = s["x"][a:a + 512].double(), s["labels"][a:a + 512]
            seen = y != -100
            z = (x @ w.T) * c["scale"]
            z = cap * torch.tanh(z / cap) if cap else z
            lse = torch.logsumexp(z, 1)
            target = torch.full_like(z, eps / v)
            target[seen, y[seen]] += 1.0 - eps
            loss.append(torch.where(seen, lse - (target * z).sum(1), 0.0))
            lses.append(torch.where(seen, lse, 0.0))
            if c["grad"]:
                d = torch.softmax(z, 1) - target
                d = d * (1.0 - (z / cap) ** 2) if cap else d
                grads.append((d * (seen * c["scale"] / count)[:, None]) @ w)
        out = {"total": torch.cat(loss).sum() / count, "loss": torch.cat(loss), "lse": torch.cat(lses)}
        if c["grad"]:
            out["dx"] = torch.cat(grads)
        return out
    if c["op"] == "clip":
        g = s["flat"].double()
        norm = torch.linalg.vector_norm(g, ord=float(c["norm"]))
        return {"norm": norm, "clipped": g * min(1.0, s["max_norm"] / (float(norm) + 1e-6))}
    sq = s["known"].double() if s["known"] is not None else \
        torch.linalg.vector_norm(torch.cat([t.double() for t in s["grads"]], 1), dim=1) ** 2
    keep = torch.minimum(torch.ones_like(sq), s["max_norm"] / torch.sqrt(sq)) / c["n"]
    return {"sums": [keep @ t.double() for t in s["grads"]], "sq_norms": sq}
