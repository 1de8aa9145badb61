"""Python binding of ``include/lora_gb300.h`` (ctypes).

Argument marshalling only: tensors are checked for dtype/contiguity/device, their
pointers and the current CUDA stream are passed to the C ABI, and status codes
become exceptions.  Every step of the computation runs in the library's kernels;
there is no fallback, and a missing library raises.

Adapters are passed as ``(W, A, B)`` tuples of bf16 CUDA tensors: W [out, in],
A [r, in], B [out, r].  Activations are token-major [M, features].
"""

from __future__ import annotations

import bisect
import ctypes
import os
import struct
import threading

import torch

from . import build as _build

ACT = {"swiglu": 0, "geglu_tanh": 1, "geglu_erf": 2}
KIND_NAMES = {0: "pack", 1: "reduce", 2: "rank_proj", 3: "rank_grad", 4: "gate_up",
              5: "proj", 6: "act_bwd", 7: "dgrad", 8: "rope", 9: "cache", 10: "attn", 11: "norm", 12: "loss",
              13: "clip"}
LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}
KV_FORMAT = {torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}
NORM_FORMAT = {"bf16": 0, "fp8": 1}
LIST_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
GRAD_NORM = {2.0: 0, float("inf"): 1}
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


class LoraCe(ctypes.Structure):
    _fields_ = [("logit_scale", ctypes.c_float), ("softcap", ctypes.c_float), ("smoothing", ctypes.c_float),
                ("reduction", ctypes.c_int), ("ignore_index", ctypes.c_int64)]


class LoraTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("count", ctypes.c_int64), ("dtype", ctypes.c_int)]


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
    "lora_rms_norm": (_INT, [_I64, _INT, _VP, _VP, _VP, _F32, _F32, _INT, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "lora_rms_norm_workspace_bytes": (_SZ, [_I64, _I64, _INT]),
    "lora_rms_norm_backward": (_INT, [_I64, _INT, _VP, _VP, _VP, _F32, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "lora_linear_ce_workspace_bytes": (_SZ, [_I64, _I64, _I64, _VP, _INT]),
    "lora_linear_ce": (_INT, [_I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "lora_scale_rows": (_INT, [_I64, _I64, _VP, _VP, _INT, _VP, _VP, _SZ, _VP]),
    "lora_grad_norm_workspace_bytes": (_SZ, [_I64]),
    "lora_grad_norm": (_INT, [_I64, _VP, _INT, _VP, _VP, _SZ, _VP]),
    "lora_clip_grads": (_INT, [_I64, _VP, _VP, _INT, _F32, _VP, _VP, _SZ, _VP]),
    "lora_clip_examples_workspace_bytes": (_SZ, [_I64, _I64]),
    "lora_clip_examples": (_INT, [_I64, _VP, _I64, _VP, _F32, _F32, _VP, _INT, _VP, _SZ, _VP]),
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


# ------------------------------------------------------------------ norm, loss, clipping

def _rows(t, name):
    """Rows [tokens, dim], or a view of heads [tokens, heads, dim], as a lora_heads_t (bytes)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        return _heads(t, name)
    if t.dtype is not _BF16 or not t.is_cuda:
        _bad_heads(t, name)
    n, dim = t.shape
    ts, one = t.stride()
    if one != 1 and dim > 1:
        _bad_heads(t, name)
    return _PACK_HEADS(t.data_ptr(), 1, ts if n > 1 else dim, dim)


def _weight(w, dim, name="weight"):
    if isinstance(w, torch.Tensor) and w.shape != (dim,):
        raise ValueError(f"{name} must be [{dim}] (got {tuple(w.shape)})")
    return _dev(w, name)


def rms_norm(x, weight, *, residual=None, eps=1e-6, offset=0.0, format="bf16", training=False, sum_out=None, out=None,
             ws=None):
    """RMS norm of the rows of x [tokens, dim] (or of the heads of a view [tokens, heads, dim]), after adding
    the residual if there is one.  Returns (y, s, rstd): s = x + residual in bf16 (x itself without one; sum_out,
    which may be x or residual, receives it), y = s * rstd * (weight + offset) in bf16, or with format "fp8" the
    pair (e4m3 codes, f32 scale of each row); rstd, f32, is what the gradient needs (None unless training)."""
    lib = _LIB or load()
    view = _rows(x, "x")
    shape = x.shape
    tokens, dim = shape[0], shape[-1]
    w_at = _weight(weight, dim)
    dev = x.device
    res = total = None
    if residual is not None:
        if residual.shape != shape:
            raise ValueError("residual must have x's shape")
        res = _rows(residual, "residual")
        if sum_out is None:
            sum_out = torch.empty(shape, dtype=_BF16, device=dev)
        elif sum_out.shape != shape:
            raise ValueError("sum_out must have x's shape")
        total = _rows(sum_out, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out receives x + residual: there is no residual")
    code = NORM_FORMAT.get(format)
    if code is None:
        raise ValueError(f"format must be one of {', '.join(NORM_FORMAT)} (got {format!r})")
    scale = None if code == 0 else torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    dtype = _BF16 if code == 0 else torch.float8_e4m3fn
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    elif out.shape != shape or out.dtype != dtype or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dtype} tensor of x's shape")
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev) if training else None
    _together(x, weight, residual, sum_out, out, ws)
    stream, wp, wn = _call(x, 256, ws)
    _check(lib.lora_rms_norm(tokens, dim, view, res, w_at, offset, eps, code, total, out.data_ptr(),
                             None if scale is None else scale.data_ptr(), None if rstd is None else rstd.data_ptr(),
                             wp, wn, stream), "lora_rms_norm")
    return (out if scale is None else (out, scale)), (x if residual is None else sum_out), rstd


def rms_norm_backward(dy, s, weight, rstd, *, offset=0.0, ds=None, dweight=True, dx=None, ws=None):
    """(dx, dweight) of rms_norm from dy, the gradient of y, and ds, the gradient that reaches s from elsewhere
    (or None).  s and rstd are the forward's.  dx (bf16, dense; may be passed in, dy or ds among others) is the
    gradient of x and of the residual; dweight is bf16 [dim], or None where it is not asked for."""
    lib = _LIB or load()
    view = _rows(s, "s")
    shape = s.shape
    tokens, dim, heads = shape[0], shape[-1], shape[1] if len(shape) == 3 else 1
    w_at = _weight(weight, dim)
    if dy.shape != shape or (ds is not None and ds.shape != shape):
        raise ValueError("dy and ds must have s's shape")
    if dx is None:
        dx = torch.empty(shape, dtype=_BF16, device=s.device)
    elif dx.shape != shape:
        raise ValueError("dx must have s's shape")
    dw = torch.empty(dim, dtype=_BF16, device=s.device) if dweight else None
    _together(s, dy, weight, rstd, ds, dx, ws)
    stream, wp, wn = _call(s, lib.lora_rms_norm_workspace_bytes(tokens, heads, dim), ws)
    _check(lib.lora_rms_norm_backward(tokens, dim, _rows(dy, "dy"), view, w_at, offset,
                                      _ints(rstd, torch.float32, shape[:-1], "rstd"),
                                      None if ds is None else _rows(ds, "ds"), _dev(dx, "dx"),
                                      None if dw is None else dw.data_ptr(), wp, wn, stream), "lora_rms_norm_backward")
    return dx, dw


def linear_cross_entropy(x, W, labels, *, scale=1.0, softcap=0.0, smoothing=0.0, ignore_index=-100, reduction="mean",
                         grad=True, dx=None, ws=None):
    """Cross entropy of the logits scale * x W^T (softcap > 0: capped by a tanh) of a frozen head W [vocab, h] over
    x [tokens, h], with int64 labels [tokens], and its gradient, without keeping the logits.  Returns (total, loss,
    lse, dx): total f32 (0-dim), the mean over the labelled tokens or the "sum"; loss and lse f32 [tokens] (0 where
    the label is ignore_index); dx the gradient of total with respect to x, or None without grad."""
    lib = _LIB or load()
    if x.dim() != 2 or W.dim() != 2 or W.shape[1] != x.shape[1]:
        raise ValueError("x must be [tokens, h] and W [vocab, h]")
    tokens, h = x.shape
    vocab, dev = W.shape[0], x.device
    if reduction not in ("mean", "sum"):
        raise ValueError('reduction must be "mean" or "sum"')
    opts = LoraCe(scale, softcap, smoothing, 1 if reduction == "mean" else 0, ignore_index)
    e = lambda *sh: torch.empty(sh, dtype=torch.float32, device=dev)  # noqa: E731
    total, loss, lse = e(), e(tokens), e(tokens)
    if not grad:
        dx = None
    elif dx is None:
        dx = torch.empty(tokens, h, dtype=_BF16, device=dev)
    elif dx.shape != x.shape:
        raise ValueError("dx must have x's shape")
    args = (_dev(x, "x"), _dev(W, "W"), _ints(labels, torch.int64, (tokens,), "labels"))
    _together(x, W, labels, dx, ws)
    need = lib.lora_linear_ce_workspace_bytes(tokens, h, vocab, _at(opts), int(grad))
    stream, wp, wn = _call(x, need, ws)
    _check(lib.lora_linear_ce(tokens, h, vocab, *args, _at(opts), loss.data_ptr(), lse.data_ptr(), total.data_ptr(),
                              _opt(dx, "dx"), wp, wn, stream), "lora_linear_ce")
    return total, loss, lse, dx


def scale_rows(x, g, *, out=None, ws=None):
    """g * x of bf16 rows [tokens, h], rounded once: g f32, 0-dim (one factor for all) or [tokens].  out may be x."""
    lib = _LIB or load()
    if x.dim() != 2:
        raise ValueError("x must be [tokens, h]")
    tokens, h = x.shape
    if out is None:
        out = torch.empty(tokens, h, dtype=_BF16, device=x.device)
    elif out.shape != x.shape:
        raise ValueError("out must have x's shape")
    args = (_dev(x, "x"), _ints(g, torch.float32, () if g.dim() == 0 else (tokens,), "g"), int(g.dim() != 0), _dev(out, "out"))
    _together(x, g, out, ws)
    stream, wp, wn = _call(x, 256, ws)
    _check(lib.lora_scale_rows(tokens, h, *args, wp, wn, stream), "lora_scale_rows")
    return out


# Whether tensors are at the addresses they had: one call for all, where this PyTorch has it.
_same_addresses = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal", None) or \
    (lambda tensors, addresses, _: list(map(torch.Tensor.data_ptr, tensors)) == addresses)


class TensorList:
    """The tensors of a call that takes many: contiguous bf16 or f32 tensors on one device, in an order
    that stays.  A program whose gradients stay the same tensors builds it once: it keeps their addresses and
    compares them at each call, so that a tensor that was given other memory (t.data = ..., set_, resize_) is
    looked over again.  A gradient that is a new tensor at each step (zero_grad(set_to_none=True), the default)
    is not the one in the list; pass such gradients as they are."""

    def __init__(self, tensors, *, kept=True):
        self.tensors = tuple(tensors)
        self._kept = kept
        self._look()

    def _look(self):
        flat = []
        for i, t in enumerate(self.tensors):
            if not isinstance(t, torch.Tensor):
                raise TypeError("a list's entries must be torch.Tensors")
            dtype = LIST_DTYPE.get(t.dtype)
            if dtype is None or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"a list's tensors must be contiguous bf16 or f32 CUDA tensors (entry {i}: {t.dtype}, "
                                 f"{t.device}, strides {t.stride()})")
            if t.get_device() != self.tensors[0].get_device():
                raise ValueError("a list's tensors must be on one device")
            flat += (t.data_ptr(), t.numel(), dtype)
        self._bytes = _pack_tensors(flat)
        self._examples = None
        if self._kept:
            # (memory that is held is not given to other tensors: an address that is the same is the same memory)
            self._memory = [t.untyped_storage() for t in self.tensors]
            self._compared = list(self.tensors), flat[::3], list(range(len(self.tensors)))
        self._spans = sorted((t.data_ptr(), t.data_ptr() + t.nbytes, i) for i, t in enumerate(self.tensors) if t.numel())
        self.overlap = any(a[1] > b[0] for a, b in zip(self._spans, self._spans[1:]))
        self._apart = None

    def __len__(self):
        return len(self.tensors)

    def _check_output(self, grads, in_place):
        """Refuses a list of outputs that overlap each other or the gradients, but (in_place) for the one in their
        own place."""
        if self.overlap:
            raise ValueError("tensors that are written overlap")
        if self._apart == (grads._bytes, in_place):      # the same addresses and sizes as at the last call
            return
        starts = [a for a, _, _ in self._spans]
        for a, z, i in grads._spans if self._meets(grads) else ():
            for own in self._spans[max(bisect.bisect_right(starts, a) - 1, 0):bisect.bisect_left(starts, z)]:
                if own[1] > a and not (in_place and own == (a, z, i)):
                    raise ValueError(f"an output overlaps a gradient that is not its own (entries {own[2]} and {i})")
        self._apart = grads._bytes, in_place

    def _meets(self, other):
        """Whether the two lists' memory reaches into each other's at all: two buffers' parts do not."""
        if not self._spans or not other._spans:
            return False
        return self._spans[0][0] < max(z for _, z, _ in other._spans) and other._spans[0][0] < max(z for _, z, _ in self._spans)

    def _example_layout(self):
        """(examples, shapes, sizes, starts, cut, total): one example's parts as one f32 buffer, each 16-byte
        aligned; cut: the lengths that cut the buffer at the parts' starts and ends, and which of them are parts."""
        if self._examples is None:
            n = self.tensors[0].shape[0] if self.tensors and self.tensors[0].dim() else 0
            if not n or any(g.dim() < 1 or g.shape[0] != n for g in self.tensors):
                raise ValueError("gradients of examples: each tensor [examples, ...], of the same examples and one at least")
            shapes = [g.shape[1:] for g in self.tensors]
            sizes = [g.numel() // n for g in self.tensors]
            starts, pieces, parts, total = [], [], [], 0
            for k in sizes:
                starts.append(total)
                parts.append(len(pieces))
                pieces += (k, -k % 4) if k % 4 else (k,)
                total += k + -k % 4
            pieces.append(n)
            self._examples = n, shapes, sizes, starts, (pieces, parts), total
        return self._examples


def _pack_tensors(flat):
    """lora_tensor_t array (bytes) of (address, count, type) after (address, count, type) ..."""
    return struct.pack("=" + "QqQ" * (len(flat) // 3), *flat)      # (the type's int and its padding: little-endian)


def tensor_list(tensors) -> TensorList:
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def _list(tensors) -> TensorList:
    """The list of a call, as its tensors lie now."""
    if not isinstance(tensors, TensorList):
        return TensorList(tensors, kept=False)
    if tensors._kept and not _same_addresses(*tensors._compared):
        tensors._look()
    return tensors


def _list_device(grads):
    """A tensor of the list's device, or of the current one for an empty list."""
    return grads.tensors[0] if grads.tensors else torch.empty(0, device=torch.device("cuda", _current_device()))


def _norm_type(norm_type) -> int:
    code = GRAD_NORM.get(float(norm_type))
    if code is None:
        raise ValueError(f"norm_type must be 2 or infinity (got {norm_type!r})")
    return code


def grad_norm(grads, *, norm_type=2.0, ws=None):
    """The norm of all gradients together (a TensorList, or any iterable of tensors), f32, 0-dim: norm_type 2
    or infinity."""
    lib = _LIB or load()
    grads = _list(grads)
    t = _list_device(grads)
    _together(t, ws)
    norm = torch.empty((), dtype=torch.float32, device=t.device)
    stream, wp, wn = _call(t, lib.lora_grad_norm_workspace_bytes(len(grads)), ws)
    _check(lib.lora_grad_norm(len(grads), grads._bytes, _norm_type(norm_type), norm.data_ptr(), wp, wn, stream),
           "lora_grad_norm")
    return norm


def clip_grad_norm(grads, max_norm, *, norm_type=2.0, out=None, ws=None):
    """Scales all gradients by min(1, max_norm / (norm + 1e-6)), in place or into out (a list of the same shapes and
    types).  Returns their norm before that, f32, 0-dim.  What is written must not overlap: a gradient twice in the
    list would be scaled twice; an output may be its own gradient, but overlap no other."""
    lib = _LIB or load()
    grads = _list(grads)
    t = _list_device(grads)
    out = None if out is None else _list(out)
    if out is None:
        if grads.overlap:
            raise ValueError("tensors that are written overlap")
    else:
        out._check_output(grads, True)
        if len(out) != len(grads):                   # (sizes and types are compared in the library)
            raise ValueError("out must match the gradients, tensor by tensor")
        if out.tensors:
            _together(t, out.tensors[0])
    _together(t, ws)
    norm = torch.empty((), dtype=torch.float32, device=t.device)
    stream, wp, wn = _call(t, lib.lora_grad_norm_workspace_bytes(len(grads)), ws)
    _check(lib.lora_clip_grads(len(grads), grads._bytes, None if out is None else out._bytes, _norm_type(norm_type),
                               max_norm, norm.data_ptr(), wp, wn, stream), "lora_clip_grads")
    return norm


def clip_examples(grads, max_norm, *, sq_norms=None, scale=1.0, out=None, ws=None):
    """DP-SGD's clipped sum: grads are tensors [examples, ...] of per-example gradients (mlp_backward_per_example's, of
    any number of calls); returns (sums, sq_norms) with sums[i] = scale * sum_e min(1, max_norm / |example e|)
    grads[i][e], f32.  sq_norms, f32 [examples]: the squared norms if they are known (mlp_backward_per_example's, added
    up), else computed.  out: the f32 tensors for sums."""
    lib = _LIB or load()
    grads = _list(grads)
    n, shapes, sizes, starts, (pieces, parts), total = grads._example_layout()
    first = grads.tensors[0]
    dev = first.device
    if out is None:
        flat = torch.empty(total + n, dtype=torch.float32, device=dev)     # (the norms behind them)
        base = flat.data_ptr()
        cut = flat.split_with_sizes(pieces)
        sums = [cut[i] if len(sh) == 1 else cut[i].view(sh) for i, sh in zip(parts, shapes)]
        packed = _pack_tensors([v for a, k in zip(starts, sizes) for v in (base + 4 * a, k, 1)])
    else:
        out = _list(out)
        if len(out) != len(grads) or any(o.shape != sh or o.dtype != torch.float32 for o, sh in zip(out.tensors, shapes)):
            raise ValueError("out must be f32 tensors of one example's shapes")
        out._check_output(grads, False)
        sums, packed = list(out.tensors), out._bytes
    given = sq_norms is not None
    if not given:
        sq_norms = cut[-1] if out is None else torch.empty(n, dtype=torch.float32, device=dev)
    sq_at = _ints(sq_norms, torch.float32, (n,), "sq_norms")
    if given and out is not None and any(a < sq_at + 4 * n and z > sq_at for a, z, _ in out._spans):
        raise ValueError("an output overlaps sq_norms")
    _together(first, sums[0], sq_norms, ws)
    stream, wp, wn = _call(first, lib.lora_clip_examples_workspace_bytes(len(grads), n), ws)
    _check(lib.lora_clip_examples(len(grads), grads._bytes, n, packed, max_norm, scale, sq_at, int(given), wp, wn, stream),
           "lora_clip_examples")
    return sums, sq_norms
