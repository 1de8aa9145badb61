"""Python binding of ``include/lora_gb300.h`` (ctypes).

Argument marshalling only: tensors are checked for dtype/contiguity/device, their
pointers and the current CUDA stream are passed to the C ABI, and status codes
become exceptions.  Every step of the computation runs in the library's kernels;
there is no fallback, and a missing library raises.

Adapters are passed as ``(W, A, B)`` tuples of bf16 CUDA tensors: W [out, in],
A [r, in], B [out, r].  Activations are token-major [M, features].
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

from . import build as _build

ACT = {"swiglu": 0, "geglu_tanh": 1, "geglu_erf": 2}
KIND_NAMES = {0: "pack", 1: "reduce", 2: "rank_proj", 3: "rank_grad", 4: "gate_up",
              5: "proj", 6: "act_bwd", 7: "dgrad", 8: "rope", 9: "cache", 10: "attn"}
LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}
KV_FORMAT = {torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}
KV_DTYPE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}
STATUS = {0: "ok", 1: "invalid argument", 2: "alignment", 3: "unsupported",
          4: "workspace too small", 5: "CUDA error", 6: "timeout", 7: "device input out of range"}


class LoraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _LIB.lora_status_string(status).decode() if _LIB is not None else STATUS.get(status, "?")
        super().__init__(f"{where}: {msg} (status {status})")


class LoraLinear(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p)]


class LoraGrads(ctypes.Structure):
    _fields_ = [("dA", ctypes.c_void_p), ("dB", ctypes.c_void_p)]


class LoraRope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("n_pos", ctypes.c_int64), ("head_dim", ctypes.c_int)]


class LoraHeads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class LoraRotary(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("n_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int), ("layout", ctypes.c_int)]


class LoraRopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("magnitude", ctypes.c_double)]


class LoraKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("format", ctypes.c_int)]


class LoraPagedBatch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int64), ("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int64),
                ("kv_len", ctypes.c_void_p), ("cu_q", ctypes.c_void_p)]


_LIB = None
_LOCK = threading.Lock()
_I64, _INT, _F32, _VP, _SZ = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t

_SIGS = {
    "lora_linear_saved_bytes": (_SZ, [_I64, _I64, _I64, _INT]),
    "lora_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64, _INT]),
    "lora_linear_forward": (_INT, [_I64, _I64, _I64, _INT, _F32, _VP, LoraLinear, _VP, _VP, _VP, _SZ, _VP]),
    "lora_linear_backward": (_INT, [_I64, _I64, _I64, _INT, _F32, _VP, LoraLinear, _VP, _VP, _VP, LoraGrads,
                                    _VP, _SZ, _VP]),
    "lora_linear_forward_noalloc": (_INT, [_I64, _I64, _I64, _INT, _F32, _VP, LoraLinear, _VP, _VP]),
    "lora_mlp_saved_bytes": (_SZ, [_I64, _I64, _I64, _INT]),
    "lora_mlp_workspace_bytes": (_SZ, [_I64, _I64, _I64, _INT]),
    "lora_mlp_forward": (_INT, [_I64, _I64, _I64, _INT, _F32, _INT, _VP, LoraLinear, LoraLinear, LoraLinear,
                                _VP, _VP, _VP, _SZ, _VP]),
    "lora_mlp_backward": (_INT, [_I64, _I64, _I64, _INT, _F32, _INT, _VP, LoraLinear, LoraLinear, LoraLinear,
                                 _VP, _VP, _VP, LoraGrads, LoraGrads, LoraGrads, _VP, _SZ, _VP]),
    "lora_mlp_per_example_workspace_bytes": (_SZ, [_I64, _I64, _I64, _INT, _I64]),
    "lora_mlp_backward_per_example": (_INT, [_I64, _I64, _I64, _INT, _F32, _INT, _I64, _VP, LoraLinear, LoraLinear,
                                             LoraLinear, _VP, _VP, _VP, LoraGrads, LoraGrads, LoraGrads, _VP, _VP,
                                             _SZ, _VP]),
    "lora_qkvo_saved_bytes": (_SZ, [_I64, _I64, _I64, _I64, _INT]),
    "lora_qkvo_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _INT]),
    "lora_rope_table": (_INT, [_VP, _VP, _I64, _INT, ctypes.c_double, _VP]),
    "lora_qkvo_forward": (_INT, [_I64, _I64, _I64, _I64, _INT, _F32, _VP, LoraLinear, LoraLinear, LoraLinear,
                                 _VP, _VP, _VP, _VP, LoraLinear, _VP, _VP, ctypes.POINTER(LoraRope), _VP, _VP,
                                 _SZ, _VP]),
    "lora_qkvo_backward": (_INT, [_I64, _I64, _I64, _I64, _INT, _F32, _VP, LoraLinear, LoraLinear, LoraLinear,
                                  _VP, LoraLinear, _VP, ctypes.POINTER(LoraRope), _VP, _VP, _VP, _VP, _VP, _VP,
                                  LoraGrads, LoraGrads, LoraGrads, LoraGrads, _VP, _SZ, _VP]),
    "lora_rotary": (_INT, [_I64, _INT, _VP, _VP, _VP, _VP, _VP, _INT, _VP, _SZ, _VP]),
    "lora_rope_table_scaled": (_INT, [_VP, _VP, _I64, _INT, ctypes.c_double, _VP, _VP]),
    "lora_kv_append": (_INT, [_I64, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "lora_kv_read": (_INT, [_I64, _I64, _VP, _VP, _I64, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "lora_paged_attention_workspace_bytes": (_SZ, [_I64, _I64, _INT, _VP]),
    "lora_paged_attention": (_INT, [_I64, _INT, _VP, _VP, _VP, _F32, _INT, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "lora_poll_status": (_INT, [_VP, _VP]),
    "lora_status_string": (ctypes.c_char_p, [_INT]),
    "lora_launch_count": (ctypes.c_uint64, []),
    "lora_set_wait_timeout": (_INT, [ctypes.c_uint64]),
    "lora_wait_timeout": (ctypes.c_uint64, []),
    "lora_test_expire_waits": (_INT, [_INT]),
    "lora_set_split_tail": (_INT, [_INT]),
    "lora_split_tail": (_INT, []),
    "lora_trace_enable": (_INT, [_INT]),
    "lora_trace_kinds": (None, [ctypes.c_uint]),
    "lora_trace_read": (_INT, [ctypes.POINTER(_INT), ctypes.POINTER(_F32), _INT]),
}
EXPORTS = tuple(_SIGS)


def load(path: str | None = None):
    """Loads the library (built in-tree by ``rank_mlp_gb300.build``); raises if absent."""
    global _LIB
    with _LOCK:
        if _LIB is not None:
            return _LIB
        path = path or _build.lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m rank_mlp_gb300.build` "
                               "(there is no fallback path)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
        return lib


def _check(status: int, where: str):
    if status != 0:
        raise LoraError(status, where)


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor (got {t.dtype}, {t.device})")
    return t.data_ptr()


def _opt(t, name):
    return None if t is None else _dev(t, name)


def _lin(lin, name) -> LoraLinear:
    W, A, B = lin
    return LoraLinear(_dev(W, name + ".W"), _dev(A, name + ".A"), _dev(B, name + ".B"))


# ------------------------------------------------------------------ workspaces

_WS = {}           # (device, stream): its workspace
_RECORDED = {}     # (device, stream): its workspaces that calls under capture were given
_capturing = torch.cuda.is_current_stream_capturing


def workspace(nbytes: int, device) -> torch.Tensor:
    """A workspace of at least nbytes for the current stream of `device` (cached per
    device and stream, grown on demand, first 256 bytes zeroed: they hold the
    asynchronous status word).  Calls that share a workspace must not overlap on the
    GPU, so each stream gets its own; calls on one stream are ordered anyway.  One that a
    graph has recorded is never freed: the graph's replays go on writing to it."""
    device = torch.device(device)
    idx = device.index if device.index is not None else torch.cuda.current_device()
    key = (idx, torch.cuda.current_stream(idx).cuda_stream)
    ws = _WS.get(key)
    if ws is None or ws.numel() < nbytes:
        old = ws
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=torch.device("cuda", idx))
        if old is not None:
            ws[:4].copy_(old[:4])     # keep a status bit that has not been polled yet (same stream)
        _WS[key] = ws
    if _capturing():
        kept = _RECORDED.setdefault(key, [])
        if not any(w is ws for w in kept):
            kept.append(ws)
    return ws


def poll_status(ws: torch.Tensor | None = None) -> int:
    """Reads and clears the status word of ws, or of the current stream's workspaces: the
    cached one and those that graphs captured on the stream have recorded."""
    lib = load()
    if ws is not None:
        return lib.lora_poll_status(ctypes.c_void_p(ws.data_ptr()), _stream(ws.device))
    ws = workspace(256, torch.cuda.current_device())
    key = (ws.get_device(), torch.cuda.current_stream(ws.device).cuda_stream)
    every = [ws] + [w for w in _RECORDED.get(key, ()) if w is not ws]
    codes = [lib.lora_poll_status(ctypes.c_void_p(w.data_ptr()), _stream(w.device)) for w in every]
    return min((c for c in codes if c), default=0)       # an expired wait before a bad input


def poll_noalloc_status() -> int:
    """Reads and clears the status word of lora_linear_forward_noalloc's scratch on the
    current device (lora_poll_status with ws = NULL); syncs the current stream."""
    return load().lora_poll_status(None, _stream(torch.cuda.current_device()))


def launch_count() -> int:
    return int(load().lora_launch_count())


def set_wait_timeout(ns: int):
    """Limit of the kernels' bounded waits, in ns (0 = the default of 2 s)."""
    _check(load().lora_set_wait_timeout(ns), "lora_set_wait_timeout")


def wait_timeout() -> int:
    return int(load().lora_wait_timeout())


def set_split_tail(mode: int):
    """Split-tail mode of the projection GEMMs: 0 automatic, 1 never, 2..4 every tail
    in that many pieces."""
    _check(load().lora_set_split_tail(mode), "lora_set_split_tail")


def split_tail() -> int:
    return int(load().lora_split_tail())


def test_expire_waits(launches: int):
    """Failure-path tests: the next `launches` GEMM or attention launches let a bounded wait expire."""
    _check(load().lora_test_expire_waits(launches), "lora_test_expire_waits")


def trace_kinds(names=None):
    """Trace only these kinds (names of KIND_NAMES; None: all)."""
    if names is None:
        mask = 0xFFFFFFFF
    else:
        inv = {v: k for k, v in KIND_NAMES.items()}
        mask = 0
        for n in names:
            mask |= 1 << inv[n]
    load().lora_trace_kinds(mask)


def trace_enable(capacity: int):
    _check(load().lora_trace_enable(capacity), "lora_trace_enable")


def trace_read(max_entries: int = 4096):
    """[(kind name, ms)] of the launches recorded since the trace was (re)started."""
    kinds = (_INT * max_entries)()
    ms = (_F32 * max_entries)()
    n = load().lora_trace_read(kinds, ms, max_entries)
    if n < 0:
        raise LoraError(5, "lora_trace_read")
    return [(KIND_NAMES.get(kinds[j], str(kinds[j])), float(ms[j])) for j in range(n)]


# ------------------------------------------------------------------ single linear

def linear_forward(x, lin, s, *, y=None, saved=None, training=True, ws=None):
    lib = load()
    W, A, B = lin
    M, fin = x.shape
    fout, r = W.shape[0], A.shape[0]
    if y is None:
        y = torch.empty(M, fout, dtype=torch.bfloat16, device=x.device)
    if saved is None and training:
        saved = torch.empty(max(lib.lora_linear_saved_bytes(M, fin, fout, r), 256), dtype=torch.uint8,
                            device=x.device)
    need = lib.lora_linear_workspace_bytes(M, fin, fout, r)
    ws = workspace(need, x.device) if ws is None else ws
    _check(lib.lora_linear_forward(M, fin, fout, r, s, _dev(x, "x"), _lin(lin, "lin"), _dev(y, "y"),
                                   None if saved is None else saved.data_ptr(), ws.data_ptr(), ws.numel(),
                                   _stream(x.device)), "lora_linear_forward")
    return y, saved


def linear_forward_noalloc(x, lin, s, *, y=None):
    """Inference forward through lora_linear_forward_noalloc: the library allocates
    nothing and the caller passes no workspace (the library's fixed scratch is used)."""
    lib = load()
    W, A, B = lin
    M = x.shape[0]
    if y is None:
        y = torch.empty(M, W.shape[0], dtype=torch.bfloat16, device=x.device)
    _check(lib.lora_linear_forward_noalloc(M, x.shape[1], W.shape[0], A.shape[0], s, _dev(x, "x"),
                                           _lin(lin, "lin"), _dev(y, "y"), _stream(x.device)),
           "lora_linear_forward_noalloc")
    return y


def linear_backward(x, lin, s, saved, dy, *, dx=None, dA=None, dB=None, ws=None):
    lib = load()
    W, A, B = lin
    M, fin = x.shape
    fout, r = W.shape[0], A.shape[0]
    dev = x.device
    dx = torch.empty(M, fin, dtype=torch.bfloat16, device=dev) if dx is None else dx
    dA = torch.empty(r, fin, dtype=torch.bfloat16, device=dev) if dA is None else dA
    dB = torch.empty(fout, r, dtype=torch.bfloat16, device=dev) if dB is None else dB
    need = lib.lora_linear_workspace_bytes(M, fin, fout, r)
    ws = workspace(need, dev) if ws is None else ws
    _check(lib.lora_linear_backward(M, fin, fout, r, s, _dev(x, "x"), _lin(lin, "lin"), saved.data_ptr(),
                                    _dev(dy, "dy"), _dev(dx, "dx"), LoraGrads(_dev(dA, "dA"), _dev(dB, "dB")),
                                    ws.data_ptr(), ws.numel(), _stream(dev)), "lora_linear_backward")
    return dx, dA, dB


# ------------------------------------------------------------------ gated MLP

def mlp_sizes(M, h, i, r):
    lib = load()
    return lib.lora_mlp_saved_bytes(M, h, i, r), lib.lora_mlp_workspace_bytes(M, h, i, r)


def mlp_forward(x, gate, up, down, s, act="swiglu", *, y=None, saved=None, training=True, ws=None):
    """y = down(act(gate(x)) * up(x)); returns (y, saved)."""
    lib = load()
    M, h = x.shape
    i, r = gate[0].shape[0], gate[1].shape[0]
    if y is None:
        y = torch.empty(M, h, dtype=torch.bfloat16, device=x.device)
    if saved is None and training:
        saved = torch.empty(max(lib.lora_mlp_saved_bytes(M, h, i, r), 256), dtype=torch.uint8, device=x.device)
    need = lib.lora_mlp_workspace_bytes(M, h, i, r)
    ws = workspace(need, x.device) if ws is None else ws
    _check(lib.lora_mlp_forward(M, h, i, r, s, ACT[act], _dev(x, "x"), _lin(gate, "gate"), _lin(up, "up"),
                                _lin(down, "down"), _dev(y, "y"), None if saved is None else saved.data_ptr(),
                                ws.data_ptr(), ws.numel(), _stream(x.device)), "lora_mlp_forward")
    return y, saved


def mlp_backward(x, gate, up, down, s, act, saved, dy, *, dx=None, grads=None, ws=None):
    """Returns dict(dx, dA_gate, dB_gate, dA_up, dB_up, dA_down, dB_down)."""
    lib = load()
    M, h = x.shape
    i, r = gate[0].shape[0], gate[1].shape[0]
    dev = x.device
    e = lambda *sh: torch.empty(*sh, dtype=torch.bfloat16, device=dev)  # noqa: E731
    out = {"dx": e(M, h) if dx is None else dx}
    if grads is None:
        grads = {"dA_gate": e(r, h), "dB_gate": e(i, r), "dA_up": e(r, h), "dB_up": e(i, r),
                 "dA_down": e(r, i), "dB_down": e(h, r)}
    out.update(grads)
    need = lib.lora_mlp_workspace_bytes(M, h, i, r)
    ws = workspace(need, dev) if ws is None else ws
    g = lambda n: LoraGrads(_dev(out["dA_" + n], "dA_" + n), _dev(out["dB_" + n], "dB_" + n))  # noqa: E731
    _check(lib.lora_mlp_backward(M, h, i, r, s, ACT[act], _dev(x, "x"), _lin(gate, "gate"), _lin(up, "up"),
                                 _lin(down, "down"), saved.data_ptr(), _dev(dy, "dy"), _dev(out["dx"], "dx"),
                                 g("gate"), g("up"), g("down"), ws.data_ptr(), ws.numel(), _stream(dev)),
           "lora_mlp_backward")
    return out


def mlp_backward_per_example(x, gate, up, down, s, act, saved, dy, n_examples, *, norms=True, ws=None):
    """Per-example adapter gradients (DP-SGD): dict(dx, dA_gate [n, r, h], dB_gate
    [n, i, r], ..., sq_norms [n] float32 or None)."""
    lib = load()
    M, h = x.shape
    i, r = gate[0].shape[0], gate[1].shape[0]
    n = int(n_examples)
    dev = x.device
    e = lambda *sh: torch.empty(*sh, dtype=torch.bfloat16, device=dev)  # noqa: E731
    out = {"dx": e(M, h), "dA_gate": e(n, r, h), "dB_gate": e(n, i, r), "dA_up": e(n, r, h), "dB_up": e(n, i, r),
           "dA_down": e(n, r, i), "dB_down": e(n, h, r),
           "sq_norms": torch.empty(n, dtype=torch.float32, device=dev) if norms else None}
    need = lib.lora_mlp_per_example_workspace_bytes(M, h, i, r, n)
    ws = workspace(need, dev) if ws is None else ws
    g = lambda k: LoraGrads(_dev(out["dA_" + k], "dA_" + k), _dev(out["dB_" + k], "dB_" + k))  # noqa: E731
    _check(lib.lora_mlp_backward_per_example(
        M, h, i, r, s, ACT[act], n, _dev(x, "x"), _lin(gate, "gate"), _lin(up, "up"), _lin(down, "down"),
        saved.data_ptr(), _dev(dy, "dy"), _dev(out["dx"], "dx"), g("gate"), g("up"), g("down"),
        None if out["sq_norms"] is None else out["sq_norms"].data_ptr(), ws.data_ptr(), ws.numel(),
        _stream(dev)), "lora_mlp_backward_per_example")
    return out


# ------------------------------------------------------------------ Q/K/V + O

def rope_table(n_pos: int, head_dim: int, base: float = 10000.0, device="cuda"):
    """(cos, sin), f32 [n_pos, head_dim/2] on `device`: the angle p * base^(-2c/head_dim)."""
    dev = torch.device(device)
    cos = torch.empty(n_pos, head_dim // 2, dtype=torch.float32, device=dev)
    sin = torch.empty_like(cos)
    _check(load().lora_rope_table(cos.data_ptr(), sin.data_ptr(), n_pos, head_dim, float(base), _stream(dev)),
           "lora_rope_table")
    return cos, sin


def _rope(rope):
    """None, or dict(cos, sin, pos, head_dim): f32 tables [n_pos, head_dim/2] and int32
    positions [M] on the device."""
    if rope is None:
        return None
    cos, sin, pos = rope["cos"], rope["sin"], rope["pos"]
    for t, dt, name in ((cos, torch.float32, "cos"), (sin, torch.float32, "sin"), (pos, torch.int32, "pos")):
        if t.dtype != dt or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"rope {name}: contiguous {dt} on the GPU expected")
    if cos.shape != sin.shape or cos.shape[1] * 2 != rope["head_dim"]:
        raise ValueError("rope tables must be [n_pos, head_dim/2]")
    return ctypes.pointer(LoraRope(cos.data_ptr(), sin.data_ptr(), pos.data_ptr(), cos.shape[0], rope["head_dim"]))


def qkvo_forward(x, q, k, v, o_in, o, s, *, bias=None, rope=None, saved=None, training=True, ws=None,
                 outs=None):
    """q/k/v from x (skipped if x is None) and the O projection of o_in (skipped if
    o_in is None).  bias: None or the frozen q/k/v biases, one bf16 tensor
    [n_q + 2 n_kv].  rope: None or dict(cos, sin, pos, head_dim), applied to q and k.
    Returns (dict(q, k, v, o), saved)."""
    lib = load()
    ref = x if x is not None else o_in
    dev = ref.device
    M = ref.shape[0]
    h = q[0].shape[1] if x is not None else o[0].shape[0]
    nq = q[0].shape[0] if x is not None else o[0].shape[1]
    nkv = k[0].shape[0] if x is not None else 8
    r = (q if x is not None else o)[1].shape[0]
    e = lambda *sh: torch.empty(*sh, dtype=torch.bfloat16, device=dev)  # noqa: E731
    res = dict(outs or {})
    if x is not None:
        for n, w in (("q", nq), ("k", nkv), ("v", nkv)):
            res.setdefault(n, e(M, w))
    if o_in is not None:
        res.setdefault("o", e(M, h))
    if saved is None and training:
        saved = torch.empty(max(lib.lora_qkvo_saved_bytes(M, h, nq, nkv, r), 256), dtype=torch.uint8,
                            device=dev)
    need = lib.lora_qkvo_workspace_bytes(M, h, nq, nkv, r)
    ws = workspace(need, dev) if ws is None else ws
    z = LoraLinear(None, None, None)
    _check(lib.lora_qkvo_forward(
        M, h, nq, nkv, r, s, _opt(x, "x"),
        _lin(q, "q") if x is not None else z, _lin(k, "k") if x is not None else z,
        _lin(v, "v") if x is not None else z,
        _opt(res.get("q"), "yq"), _opt(res.get("k"), "yk"), _opt(res.get("v"), "yv"),
        _opt(o_in, "o_in"), _lin(o, "o") if o_in is not None else z, _opt(res.get("o"), "yo"),
        _opt(bias, "bias"), _rope(rope), None if saved is None else saved.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream(dev)),
        "lora_qkvo_forward")
    return res, saved


def qkvo_backward(x, q, k, v, o_in, o, s, saved, dyq=None, dyk=None, dyv=None, dyo=None, *, rope=None,
                  ws=None):
    """Returns dict(dx, do_in, dA_q, dB_q, ..., dA_o, dB_o) for the halves present.
    With rope (the forward's), dyq and dyk are gradients of the rotated q and k."""
    lib = load()
    ref = x if x is not None else o_in
    dev = ref.device
    M = ref.shape[0]
    h = q[0].shape[1] if x is not None else o[0].shape[0]
    nq = q[0].shape[0] if x is not None else o[0].shape[1]
    nkv = k[0].shape[0] if x is not None else 8
    r = (q if x is not None else o)[1].shape[0]
    e = lambda *sh: torch.empty(*sh, dtype=torch.bfloat16, device=dev)  # noqa: E731
    out = {}
    z = LoraGrads(None, None)
    zl = LoraLinear(None, None, None)
    if x is not None:
        out["dx"] = e(M, h)
        for n, w in (("q", nq), ("k", nkv), ("v", nkv)):
            out["dA_" + n], out["dB_" + n] = e(r, h), e(w, r)
    if o_in is not None:
        out["do_in"] = e(M, nq)
        out["dA_o"], out["dB_o"] = e(r, nq), e(h, r)
    gr = lambda n: LoraGrads(out["dA_" + n].data_ptr(), out["dB_" + n].data_ptr()) if "dA_" + n in out else z  # noqa: E731,E501
    need = lib.lora_qkvo_workspace_bytes(M, h, nq, nkv, r)
    ws = workspace(need, dev) if ws is None else ws
    _check(lib.lora_qkvo_backward(
        M, h, nq, nkv, r, s, _opt(x, "x"),
        _lin(q, "q") if x is not None else zl, _lin(k, "k") if x is not None else zl,
        _lin(v, "v") if x is not None else zl, _opt(o_in, "o_in"),
        _lin(o, "o") if o_in is not None else zl, saved.data_ptr(), _rope(rope),
        _opt(dyq, "dyq"), _opt(dyk, "dyk"), _opt(dyv, "dyv"), _opt(out.get("dx"), "dx"),
        _opt(dyo, "dyo"), _opt(out.get("do_in"), "do_in"), gr("q"), gr("k"), gr("v"), gr("o"),
        ws.data_ptr(), ws.numel(), _stream(dev)), "lora_qkvo_backward")
    return out


# ------------------------------------------------------------------ serving: rotary, cache, attention
#
# Tensors of heads are views [tokens, heads, head_dim] (bf16, feature stride 1), so that
# q, k and v can be slices of one buffer.  The structures handed to the library live
# until the call returns; the library copies what it needs.

# A call of a few microseconds on the GPU is bounded by this code, so it checks each tensor
# once, asks for the stream once, and packs the small structures as bytes (a ctypes
# Structure takes four times as long to fill).

_BF16 = torch.bfloat16
_PACK_HEADS = struct.Struct("=Q3q").pack         # lora_heads_t
_PACK_ROTARY = struct.Struct("=3Qq2i").pack      # lora_rotary_t
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda idx: torch.cuda.current_stream(idx).cuda_stream)


def _bad_heads(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise ValueError(f"{name} must be a bf16 CUDA tensor [tokens, heads, head_dim] with feature stride 1 "
                     f"(got {t.dtype}, {t.device}, {tuple(t.shape)}, strides {t.stride()})")


def _heads(t, name):
    """t as a lora_heads_t (bytes)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or not t.is_cuda or t.dim() != 3:
        _bad_heads(t, name)
    n, heads, dim = t.shape
    ts, hs, one = t.stride()
    if one != 1 and dim > 1:
        _bad_heads(t, name)
    # the stride of an extent of one says nothing; a whole row satisfies every rule
    return _PACK_HEADS(t.data_ptr(), heads, ts if n > 1 else heads * dim, hs if heads > 1 else dim)


def _ints(t, dtype, shape, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)} (got {t.dtype}, "
                         f"{t.device}, {tuple(t.shape)})")
    return t.data_ptr()


_current_device = torch.cuda.current_device


def _together(first, *others):
    """Checks that a call's tensors (None: not passed) lie on the current device, whose context
    its kernels run in: a kernel that reads another device's memory faults."""
    idx = first.get_device()
    for t in others:
        if t is not None and t.get_device() != idx:
            raise ValueError(f"tensors of one call must be on one device (got {idx} and {t.get_device()})")
    if idx != _current_device():
        raise ValueError(f"the tensors are on device {idx}, the current device is {_current_device()}")


def _rotary(rope, tokens) -> bytes:
    """A lora_rotary_t of dict(cos, sin, pos[, layout]): f32 tables [n_pos, rot_dim/2] and int32 positions
    [tokens] on the device; layout "half" (default) or "interleaved"."""
    cos = rope["cos"]
    shape = cos.shape
    if len(shape) != 2:
        raise ValueError("rope tables must be [n_pos, rot_dim/2]")
    return _PACK_ROTARY(_ints(cos, torch.float32, shape, "rope cos"),
                        _ints(rope["sin"], torch.float32, shape, "rope sin"),
                        _ints(rope["pos"], torch.int32, (tokens,), "rope pos"), shape[0], 2 * shape[1],
                        LAYOUT[rope.get("layout", "half")])


def _call(t, nbytes, ws):
    """(stream, workspace address, its bytes) of a call on t's device; ws as the caller's, or
    the current stream's cached one."""
    idx = t.get_device()
    stream = _RAW_STREAM(idx)
    if ws is None:
        ws = _WS.get((idx, stream))
        if ws is None or ws.numel() < nbytes or _capturing():
            ws = workspace(nbytes, t.device)
    return stream, ws.data_ptr(), ws.numel()


_at = ctypes.addressof


def rope_table_scaled(n_pos: int, rot_dim: int, base: float = 10000.0, scaling: dict | None = None, device="cuda"):
    """(cos, sin), f32 [n_pos, rot_dim/2]: ``rope_table`` with the frequencies scaled for a
    long context.  scaling: None, or dict(kind="linear" | "ntk" | "yarn" | "wavelength",
    factor, original_len, low, high, magnitude), the fields of lora_rope_scaling_t (low and
    high default to 1 and 32 for yarn, 1 and 4 for wavelength)."""
    sc = dict(scaling or {})
    kind = sc.pop("kind", "plain")
    low, high = sc.pop("low", 1.0), sc.pop("high", 32.0 if kind == "yarn" else 4.0)
    st = LoraRopeScaling(ROPE_SCALING[kind], sc.pop("factor", 1.0), sc.pop("original_len", 0.0), low, high,
                         sc.pop("magnitude", 0.0))
    if sc:
        raise ValueError(f"unknown rope scaling fields {sorted(sc)}")
    dev = torch.device(device)
    cos = torch.empty(n_pos, rot_dim // 2, dtype=torch.float32, device=dev)
    sin = torch.empty_like(cos)
    _check(load().lora_rope_table_scaled(cos.data_ptr(), sin.data_ptr(), n_pos, rot_dim, float(base), _at(st),
                                         _stream(dev)), "lora_rope_table_scaled")
    return cos, sin


def rotary(q, k=None, *, rope, inverse=False, q_out=None, k_out=None, ws=None):
    """Rotary positions of q and k, views [tokens, heads, head_dim], in one launch: returns
    the rotated q, or (q, k).  rope: dict(cos, sin, pos[, layout]) with tables
    [n_pos, rot_dim/2]; features from rot_dim on pass through.  inverse turns back (the
    gradient).  q_out and k_out may be q and k themselves."""
    lib = _LIB or load()
    shape = q.shape
    view = _heads(q, "q")
    tokens, dim = shape[0], shape[2]
    if q_out is None:
        q_out = torch.empty(shape, dtype=_BF16, device=q.device)
    elif q_out.shape != shape:
        raise ValueError("q_out must have q's shape")
    rot = _rotary(rope, tokens)
    _together(q, q_out, k, k_out, rope["cos"], rope["sin"], rope["pos"], ws)
    stream, wp, wn = _call(q, 256, ws)
    if k is None:
        _check(lib.lora_rotary(tokens, dim, view, _heads(q_out, "q_out"), None, None, rot, int(inverse), wp, wn, stream),
               "lora_rotary")
        return q_out
    kshape = k.shape
    if kshape[0] != tokens or kshape[2] != dim:
        raise ValueError("k must have q's tokens and head_dim")
    if k_out is None:
        k_out = torch.empty(kshape, dtype=_BF16, device=q.device)
    elif k_out.shape != kshape:
        raise ValueError("k_out must have k's shape")
    _check(lib.lora_rotary(tokens, dim, view, _heads(q_out, "q_out"), _heads(k, "k"), _heads(k_out, "k_out"), rot,
                           int(inverse), wp, wn, stream), "lora_rotary")
    return q_out, k_out


class KVCache:
    """A paged cache of K and V over tensors that the caller owns: k, v [n_pages, heads,
    page_size, head_dim] (bf16, float8_e4m3fn or int8) and, for the 8-bit formats, their
    scales k_scale, v_scale, f32 [n_pages, heads, page_size].  Slot s is row s % page_size
    of page s // page_size."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.dtype not in KV_FORMAT:
            raise ValueError("cache pages must be [n_pages, heads, page_size, head_dim] of bf16, float8_e4m3fn or int8")
        shape = tuple(k.shape)
        scaled = k.dtype != torch.bfloat16
        if scaled != (k_scale is not None) or scaled != (v_scale is not None):
            raise ValueError("scales belong to the 8-bit formats, and to both K and V")
        sc = [_ints(t, torch.float32, shape[:3], n) if scaled else None
              for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale"))]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.heads, self.page_size, self.head_dim = shape
        self._struct = LoraKvCache(_ints(k, k.dtype, shape, "k"), _ints(v, k.dtype, shape, "v"), sc[0], sc[1],
                                   shape[0], shape[2], shape[1], shape[3], KV_FORMAT[k.dtype])
        if any(t is not None and t.get_device() != k.get_device() for t in (v, k_scale, v_scale)):
            raise ValueError("a cache's tensors must be on one device")
        self._at = _at(self._struct)


def kv_cache(n_pages: int, page_size: int, heads: int, head_dim: int, format: str = "bf16", device="cuda") -> KVCache:
    """A zeroed KVCache of the given format ("bf16", "fp8" or "int8")."""
    dev = torch.device(device)
    k, v = (torch.zeros(n_pages, heads, page_size, head_dim, dtype=torch.uint8 if format != "bf16" else torch.bfloat16,
                        device=dev).view(KV_DTYPE[format]) for _ in range(2))
    scales = [None if format == "bf16" else torch.zeros(n_pages, heads, page_size, dtype=torch.float32, device=dev)
              for _ in range(2)]
    return KVCache(k, v, *scales)


def kv_append(cache: KVCache, k, v, slots, *, q=None, rope=None, q_out=None, ws=None):
    """Writes k and v (views [tokens, heads, head_dim]) to the cache's slots (int64
    [tokens]; negative: skipped).  With rope, k is rotated first, and q in the same launch:
    returns the rotated q (q_out, which may be q), or None without q."""
    lib = _LIB or load()
    shape = k.shape
    view = _heads(k, "k")
    tokens, dim = shape[0], cache.head_dim
    if shape[1] != cache.heads or shape[2] != dim or v.shape != shape:
        raise ValueError(f"k and v must be [tokens, {cache.heads}, {dim}]")
    slot_at = _ints(slots, torch.int64, (tokens,), "slots")
    rot = None if rope is None else _rotary(rope, tokens)
    _together(k, v, cache.k, slots, q, q_out, ws)
    if rope is not None:
        _together(k, rope["cos"], rope["sin"], rope["pos"])
    stream, wp, wn = _call(k, 256, ws)
    if q is None:
        _check(lib.lora_kv_append(tokens, cache._at, view, _heads(v, "v"), slot_at, None, None, rot, wp, wn, stream),
               "lora_kv_append")
        return None
    if rot is None:
        raise ValueError("q is passed to be rotated: rope is missing")
    qshape = q.shape
    if qshape[0] != tokens or qshape[2] != dim:
        raise ValueError("q must have k's tokens and head_dim")
    if q_out is None:
        q_out = torch.empty(qshape, dtype=_BF16, device=q.device)
    elif q_out.shape != qshape:
        raise ValueError("q_out must have q's shape")
    _check(lib.lora_kv_append(tokens, cache._at, view, _heads(v, "v"), slot_at, _heads(q, "q"), _heads(q_out, "q_out"),
                              rot, wp, wn, stream), "lora_kv_append")
    return q_out


def kv_read(cache: KVCache, page_table, cu_kv, total: int, *, ws=None):
    """(k, v), bf16 [total, heads, head_dim]: the sequences' cached rows one after the
    other, sequence b's at rows [cu_kv[b], cu_kv[b+1]).  page_table int32 [n_seqs,
    max_pages], cu_kv int32 [n_seqs + 1], both on the device."""
    lib = _LIB or load()
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_seqs, max_pages]")
    n, width = page_table.shape
    _together(cache.k, page_table, cu_kv, ws)
    shape, dev = (total, cache.heads, cache.head_dim), cache.k.device
    k, v = torch.empty(shape, dtype=_BF16, device=dev), torch.empty(shape, dtype=_BF16, device=dev)
    stream, wp, wn = _call(cache.k, 256, ws)
    _check(lib.lora_kv_read(n, total, cache._at, _ints(page_table, torch.int32, (n, width), "page_table"), width,
                            _ints(cu_kv, torch.int32, (n + 1,), "cu_kv"), k.data_ptr(), v.data_ptr(), wp, wn, stream),
           "lora_kv_read")
    return k, v


class PagedBatch:
    """The sequences of a step: page_table int32 [n_seqs, max_pages], kv_len int32 [n_seqs]
    (cached positions, the new tokens' own among them) and cu_q int32 [n_seqs + 1] (their
    query rows), all on the device.  One object serves all layers of a step, and later
    steps too when the tensors are updated in place."""

    def __init__(self, page_table, kv_len, cu_q):
        if page_table.dim() != 2:
            raise ValueError("page_table must be [n_seqs, max_pages]")
        n, width = page_table.shape
        self.page_table, self.kv_len, self.cu_q = page_table, kv_len, cu_q
        self._struct = LoraPagedBatch(n, _ints(page_table, torch.int32, (n, width), "page_table"), width,
                                      _ints(kv_len, torch.int32, (n,), "kv_len"),
                                      _ints(cu_q, torch.int32, (n + 1,), "cu_q"))
        if not page_table.get_device() == kv_len.get_device() == cu_q.get_device():
            raise ValueError("a batch's tensors must be on one device")
        self._at, self.n_seqs = _at(self._struct), n


def paged_batch(page_table, kv_len, cu_q) -> PagedBatch:
    return PagedBatch(page_table, kv_len, cu_q)


def paged_attention(q, cache: KVCache, batch: PagedBatch, *, scale=None, causal=True, window=0, out=None, lse=None,
                    ws=None):
    """Attention of the new tokens' q (view [tokens, heads_q, head_dim]) over the cached
    positions that each sees: out, bf16 [tokens, heads_q, head_dim].  scale defaults to
    head_dim ** -0.5; causal and window as in lora_paged_attention.  lse: None, or an f32
    [tokens, heads_q] tensor that receives the logarithm of each sum."""
    lib = _LIB or load()
    shape = q.shape
    view = _heads(q, "q")
    tokens, hq, dim = shape
    if dim != cache.head_dim:
        raise ValueError(f"q must have the cache's head_dim {cache.head_dim}")
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
        out_at = out.data_ptr()
    elif out.shape != shape:
        raise ValueError("out must have q's shape")
    else:
        out_at = _dev(out, "out")
    lse_at = None if lse is None else _ints(lse, torch.float32, (tokens, hq), "lse")
    _together(q, cache.k, batch.cu_q, out, lse, ws)
    need = lib.lora_paged_attention_workspace_bytes(tokens, batch.n_seqs, hq, cache._at)
    stream, wp, wn = _call(q, need, ws)
    _check(lib.lora_paged_attention(tokens, hq, view, cache._at, batch._at, dim ** -0.5 if scale is None else scale,
                                    int(causal), window, out_at, lse_at, wp, wn, stream), "lora_paged_attention")
    return out
