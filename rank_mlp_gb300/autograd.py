"""torch.autograd functions over the library's entry points, for training loops that
call ``loss.backward()``.

They only route tensors: the forward and backward of each function are one call each
of ``lora_mlp_forward/backward``, ``lora_qkvo_forward/backward`` (the Q/K/V half),
``lora_linear_forward/backward``, ``lora_rotary`` (both ways), ``lora_rms_norm`` and its
backward, and ``lora_linear_ce``, whose one call gives the loss and the gradient, which
``lora_scale_rows`` scales by the loss's own.  The base weights W are frozen ("Model Patches and
Kernels": a frozen weight gets no gradient), so they never receive a gradient; the
adapters A, B and the input x do.  Inputs may carry leading batch dimensions
([..., features]); every tensor is bf16 on the GPU.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding


def _flat(t: torch.Tensor) -> torch.Tensor:
    return t.reshape(-1, t.shape[-1]).contiguous()


def _bf16(t: torch.Tensor) -> torch.Tensor:
    return t if t.dtype == torch.bfloat16 else t.to(torch.bfloat16)


class LoraMLPFunction(torch.autograd.Function):
    """y = down(act(gate(x)) * up(x)), each a LoRA linear W x + s B A x."""

    @staticmethod
    def forward(ctx, x, Wg, Ag, Bg, Wu, Au, Bu, Wd, Ad, Bd, s: float, act: str = "swiglu"):
        x2 = _flat(x)
        y, saved = binding.mlp_forward(x2, (Wg, Ag, Bg), (Wu, Au, Bu), (Wd, Ad, Bd), s, act)
        ctx.save_for_backward(x2, Wg, Ag, Bg, Wu, Au, Bu, Wd, Ad, Bd, saved)
        ctx.s, ctx.act, ctx.xshape = s, act, x.shape
        return y.reshape(*x.shape[:-1], y.shape[-1])

    @staticmethod
    def backward(ctx, dy):
        x2, Wg, Ag, Bg, Wu, Au, Bu, Wd, Ad, Bd, saved = ctx.saved_tensors
        g = binding.mlp_backward(x2, (Wg, Ag, Bg), (Wu, Au, Bu), (Wd, Ad, Bd), ctx.s, ctx.act, saved,
                                 _bf16(_flat(dy)))
        return (g["dx"].reshape(ctx.xshape), None, g["dA_gate"], g["dB_gate"], None, g["dA_up"], g["dB_up"],
                None, g["dA_down"], g["dB_down"], None, None)


class LoraQKVFunction(torch.autograd.Function):
    """(q, k, v) from one input, each a LoRA linear, with optional frozen biases (one
    bf16 tensor [n_q + 2 n_kv]) and optional RoPE on q and k (dict(cos, sin, pos,
    head_dim), see ``binding.rope_table``)."""

    @staticmethod
    def forward(ctx, x, Wq, Aq, Bq, Wk, Ak, Bk, Wv, Av, Bv, s: float, bias=None, rope=None):
        x2 = _flat(x)
        out, saved = binding.qkvo_forward(x2, (Wq, Aq, Bq), (Wk, Ak, Bk), (Wv, Av, Bv), None, None, s,
                                          bias=bias, rope=rope)
        ctx.save_for_backward(x2, Wq, Aq, Bq, Wk, Ak, Bk, Wv, Av, Bv, saved)
        ctx.s, ctx.rope, ctx.xshape = s, rope, x.shape
        lead = x.shape[:-1]
        return tuple(out[n].reshape(*lead, out[n].shape[-1]) for n in ("q", "k", "v"))

    @staticmethod
    def backward(ctx, dq, dk, dv):
        x2, Wq, Aq, Bq, Wk, Ak, Bk, Wv, Av, Bv, saved = ctx.saved_tensors
        z = lambda d, W: torch.zeros(x2.shape[0], W.shape[0], dtype=torch.bfloat16, device=x2.device) \
            if d is None else _bf16(_flat(d))  # noqa: E731
        g = binding.qkvo_backward(x2, (Wq, Aq, Bq), (Wk, Ak, Bk), (Wv, Av, Bv), None, None, ctx.s, saved,
                                  z(dq, Wq), z(dk, Wk), z(dv, Wv), None, rope=ctx.rope)
        return (g["dx"].reshape(ctx.xshape), None, g["dA_q"], g["dB_q"], None, g["dA_k"], g["dB_k"],
                None, g["dA_v"], g["dB_v"], None, None, None)


class LoraLinearFunction(torch.autograd.Function):
    """y = x W^T + s (x A^T) B^T (the output projection, or any single LoRA linear)."""

    @staticmethod
    def forward(ctx, x, W, A, B, s: float):
        x2 = _flat(x)
        y, saved = binding.linear_forward(x2, (W, A, B), s)
        ctx.save_for_backward(x2, W, A, B, saved)
        ctx.s, ctx.xshape = s, x.shape
        return y.reshape(*x.shape[:-1], y.shape[-1])

    @staticmethod
    def backward(ctx, dy):
        x2, W, A, B, saved = ctx.saved_tensors
        dx, dA, dB = binding.linear_backward(x2, (W, A, B), ctx.s, saved, _bf16(_flat(dy)))
        return dx.reshape(ctx.xshape), None, dA, dB, None


class RotaryFunction(torch.autograd.Function):
    """Rotary positions of q and k (or None), views [tokens, heads, head_dim] (rope as in
    ``binding.rotary``); the gradient is the rotation back, and its gradient the rotation.
    The tables and positions are saved: a change in place before the backward is an error."""

    @staticmethod
    def forward(ctx, q, k, rope, inverse=False):
        ctx.save_for_backward(rope["cos"], rope["sin"], rope["pos"])
        ctx.layout, ctx.inverse = rope.get("layout", "half"), inverse
        ctx.set_materialize_grads(False)
        return binding.rotary(q, k, rope=rope, inverse=inverse)

    @staticmethod
    def backward(ctx, dq, dk=None):
        cos, sin, pos = ctx.saved_tensors
        rope = {"cos": cos, "sin": sin, "pos": pos, "layout": ctx.layout}
        wanted = [d for d, need in zip((dq, dk), ctx.needs_input_grad) if need and d is not None]
        back = []
        if wanted:
            back = RotaryFunction.apply(*(_rows(_bf16(d)) for d in wanted), *(None,) * (2 - len(wanted)), rope,
                                        not ctx.inverse)
            back = list(back) if len(wanted) == 2 else [back]
        grads = [back.pop(0) if need and d is not None else None for d, need in zip((dq, dk), ctx.needs_input_grad)]
        return *grads, None, None


class RmsNormFunction(torch.autograd.Function):
    """(y, s) of ``binding.rms_norm`` in bf16 with a residual, or y without one, over rows [..., dim] (or
    views of heads [tokens, heads, dim]).  The gradient that reaches s is added in the same call; a
    weight that needs no gradient gets none."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps: float, offset: float):
        x2, r2 = _tokens(x, residual)
        y, s, rstd = binding.rms_norm(x2, weight, residual=r2, eps=eps, offset=offset, training=True)
        ctx.save_for_backward(s, weight, rstd)
        ctx.offset, ctx.xshape = offset, x.shape
        ctx.set_materialize_grads(False)
        return y.reshape(x.shape) if residual is None else (y.reshape(x.shape), s.reshape(x.shape))

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        if dy is None:
            return ds if need_x else None, None, ds if need_r else None, None, None
        dx, dw = binding.rms_norm_backward(_strided(_bf16(dy).reshape(s.shape)), s, weight, rstd, offset=ctx.offset,
                                           ds=None if ds is None else _strided(_bf16(ds).reshape(s.shape)), dweight=need_w)
        dx = dx.reshape(ctx.xshape)
        return dx if need_x else None, dw, dx if need_r else None, None, None


class LinearCrossEntropyFunction(torch.autograd.Function):
    """``binding.linear_cross_entropy`` over rows [..., h] and labels [...]: the total, or with reduction
    "none" each token's loss.  The forward's call computes the gradient too, where x needs one;
    the backward scales it.  W is frozen."""

    @staticmethod
    def forward(ctx, x, W, labels, scale, softcap, smoothing, ignore_index, reduction):
        ctx.xshape, ctx.none = x.shape, reduction == "none"
        total, loss, _, dx = binding.linear_cross_entropy(
            _flat(x), W, labels.reshape(-1).contiguous(), scale=scale, softcap=softcap, smoothing=smoothing,
            ignore_index=ignore_index, reduction="sum" if ctx.none else reduction, grad=ctx.needs_input_grad[0])
        # (a mask: the labels' own buffer may hold the next batch by the time of the backward)
        ctx.save_for_backward(dx, labels == ignore_index if ctx.none and dx is not None else None)
        return loss.reshape(labels.shape) if ctx.none else total

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        dx, unlabelled = ctx.saved_tensors
        if ctx.none:
            g = torch.where(unlabelled, 0.0, g)              # (such a token has no part, whatever g says there)
        # one rounding more where g is no power of two
        dx = binding.scale_rows(dx, g.float().reshape(-1 if ctx.none else ()).contiguous())
        return dx.reshape(ctx.xshape), None, None, None, None, None, None, None


def _tokens(x, residual):
    """Both in one layout that the library takes: views of heads [tokens, heads, dim] where that saves a copy (and
    the library takes so many), else rows [tokens, dim]."""
    both = [t for t in (x, residual) if t is not None]
    if all(t.dim() == 3 for t in both) and not all(t.is_contiguous() for t in both) and x.shape[1] <= 65535:
        both = [_strided(t) for t in both]
    else:
        both = [_strided(t) if t.dim() == 2 else _flat(t) for t in both]
    return both[0], None if residual is None else both[1]


def _strided(t):
    """t, or a copy where its strides do not suit the library."""
    fits = t.stride(-1) == 1 and all(s % 8 == 0 for s in t.stride()[:-1]) and t.data_ptr() % 16 == 0
    return t if fits else t.contiguous()


def _rows(d):
    """d as a view of heads that the library takes."""
    fits = d.stride(-1) == 1 and all(s % 8 == 0 for s in d.stride()[:2]) and d.data_ptr() % 16 == 0
    return d if fits else d.contiguous()


def lora_rotary(q, k, rope):
    """(rotated q, rotated k), or the rotated q alone where k is None."""
    return RotaryFunction.apply(q, k, rope)


def lora_rms_norm(x, weight, residual=None, eps=1e-6, offset=0.0):
    """y, or with a residual (y, x + residual)."""
    return RmsNormFunction.apply(x, weight, residual, eps, offset)


def lora_linear_cross_entropy(x, W, labels, *, scale=1.0, softcap=0.0, smoothing=0.0, ignore_index=-100,
                              reduction="mean"):
    """The loss of a frozen head W over x: reduction "mean" over the labelled tokens, "sum" or "none"."""
    return LinearCrossEntropyFunction.apply(x, W, labels, scale, softcap, smoothing, ignore_index, reduction)


def lora_mlp(x, gate, up, down, s, act="swiglu"):
    """gate, up, down: (W, A, B) triples."""
    return LoraMLPFunction.apply(x, *gate, *up, *down, s, act)


def lora_qkv(x, q, k, v, s, bias=None, rope=None):
    return LoraQKVFunction.apply(x, *q, *k, *v, s, bias, rope)


def lora_linear(x, lin, s):
    return LoraLinearFunction.apply(x, *lin, s)
