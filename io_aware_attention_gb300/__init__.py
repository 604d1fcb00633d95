"""GB300 (sm_103a) IO-aware attention: Python binding of the C ABI in include/fa.h.

Only argument marshalling happens here; every step of the computation runs in
the CUDA kernels of ``libfa_gb300.so``.  There is no fallback: if the library
is missing or the device is not sm_103, calls raise.

    o, lse = io_aware_attention_gb300.fwd(q, k, v, causal=True)

q, k, v: CUDA bf16 tensors of shape (B, H, N, d), contiguous, d a multiple of
8 from 8 to 128.
Returns o (bf16, same shape) and lse (fp32, (B, H, N)), the natural-log
logsumexp of each row's scaled, masked scores.

    dq, dk, dv = io_aware_attention_gb300.bwd(q, k, v, o, lse, do, causal=True)

gives the gradients for the output gradient ``do`` (the same head sizes),
recomputing the probabilities from ``lse``.

    o, lse = io_aware_attention_gb300.decode(q, k_cache, v_cache, causal=True)

is split-KV decode of up to 8 query rows against a long cache (the same head
sizes).

    y = io_aware_attention_gb300.bias_gelu_dropout(x, bias, keep, p)

is the fused elementwise chain (bias add, tanh GELU, dropout with a packed
keep mask drawn by the caller) in one HBM read and one write.

    freqs, factor = io_aware_attention_gb300.rope_frequencies(d, base=10000.0)
    q, k = io_aware_attention_gb300.rope(q, k, freqs, factor=factor)
    dq, dk = io_aware_attention_gb300.rope_bwd(dq, dk, freqs, factor=factor)

turns queries and keys by their positions (half or interleaved pairs, all or
part of the head, any position), and gives the gradient.

    pool = io_aware_attention_gb300.qcache_pool(num_pages, Hkv, d)

is a paged cache held in 4 bits, and a decode step over it, of one token of
every sequence (grouped heads, sequences of unequal lengths), is

    q, k = io_aware_attention_gb300.rope(q, k, freqs, positions=positions, factor=factor)
    positions += 1
    lens += 1
    io_aware_attention_gb300.qcache_append(k, v, pool, table, lens)
    o, lse = io_aware_attention_gb300.qcache_decode(q, pool, table, lens)
    weights = io_aware_attention_gb300.qcache_weights(q, lse, pool, table, lens, weights)
    kept, lens, weights = io_aware_attention_gb300.qcache_evict(pool, table, lens, weights, keep)

the last line, now and then, dropping the keys that gathered the least
attention.  positions, integers (B, 1), counts the tokens of the text and lens
the keys that the cache holds: they part at the first eviction, after which kept
keys still stand, turned, where they were produced.

The ``*_into`` forms write into caller-provided tensors; their shapes, dtypes
and devices are checked here, because the C ABI sees only pointers and sizes.
Work is enqueued on ``stream``, by default the current stream, of the current
CUDA device, which must be the tensors' device (``fwd``, ``bwd`` and
``decode`` switch to it themselves).  The checks of a ``fwd_into`` call take
one pass over its tensors (a few microseconds of host time per call).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

from . import _build

__all__ = ["fwd", "fwd_into", "bwd", "bwd_into", "bwd_workspace_bytes", "bias_gelu_dropout", "decode", "decode_into", "decode_workspace_bytes", "check_device_status", "get_device_status",
           "rope", "rope_into", "rope_bwd", "rope_frequencies", "qcache_pool", "qcache_append", "qcache_read",
           "qcache_decode", "qcache_decode_into", "qcache_decode_workspace_bytes", "qcache_weights", "qcache_evict",
           "set_wait_limit_ns", "debug_skip_k_tile", "debug_set_schedule", "FaError", "library", "library_path", "version", "STATUS"]

STATUS = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_CUDA",
          4: "FA_ERR_TIMEOUT", 5: "FA_ERR_TOO_LARGE"}
EXPORTS = ["fa_fwd", "fa_bwd", "fa_bwd_workspace_bytes", "fa_bias_gelu_dropout", "fa_decode", "fa_decode_workspace_bytes", "fa_decode_static",
           "fa_rope", "fa_qcache_append", "fa_qcache_read", "fa_qcache_decode", "fa_qcache_decode_workspace_bytes",
           "fa_qcache_weights", "fa_qcache_evict", "fa_check_device_status", "fa_get_device_status",
           "fa_set_wait_limit_ns", "fa_debug_skip_k_tile", "fa_debug_set_schedule", "fa_debug_decode_plan", "fa_status_string",
           "fa_version"]


class FaError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        self.name = STATUS.get(code, f"status {code}")
        super().__init__(f"{what}: {self.name}" if what else self.name)


_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def library():
    """Load ``libfa_gb300.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as "
                           "g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float, vp]
    lib.fa_fwd.restype = ctypes.c_int
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float,
                           vp, ctypes.c_size_t, vp]
    lib.fa_bwd.restype = ctypes.c_int
    lib.fa_bwd_workspace_bytes.argtypes = [i64, i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_bwd_workspace_bytes.restype = ctypes.c_int
    lib.fa_bias_gelu_dropout.argtypes = [vp, vp, vp, vp, i64, i64, ctypes.c_float, vp]
    lib.fa_bias_gelu_dropout.restype = ctypes.c_int
    lib.fa_decode.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float, vp,
                              ctypes.c_size_t, vp]
    lib.fa_decode.restype = ctypes.c_int
    lib.fa_decode_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_decode_workspace_bytes.restype = ctypes.c_int
    lib.fa_decode_static.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float,
                                     vp]
    lib.fa_decode_static.restype = ctypes.c_int
    ci, cf, sz = ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_rope.argtypes = [vp] * 8 + [i64] * 5 + [vp, i64, ci, cf, ci, vp, ci, i64, vp, vp]
    lib.fa_rope.restype = ctypes.c_int
    lib.fa_qcache_append.argtypes = [vp] * 4 + [i64] * 4 + [cf, cf, vp, i64, vp, i64, vp, vp]
    lib.fa_qcache_append.restype = ctypes.c_int
    lib.fa_qcache_read.argtypes = [vp, i64, vp, i64, vp, vp, vp] + [i64] * 4 + [ci, cf, cf, vp]
    lib.fa_qcache_read.restype = ctypes.c_int
    lib.fa_qcache_decode.argtypes = [vp, vp, i64, vp, i64, vp, vp, vp] + [i64] * 5 + [ci, cf, cf, cf, vp, sz, vp]
    lib.fa_qcache_decode.restype = ctypes.c_int
    lib.fa_qcache_decode_workspace_bytes.argtypes = [i64] * 6 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_qcache_decode_workspace_bytes.restype = ctypes.c_int
    lib.fa_qcache_weights.argtypes = [vp, vp, vp, i64, vp, i64, vp, vp, vp] + [i64] * 6 + [ci, cf, cf, vp]
    lib.fa_qcache_weights.restype = ctypes.c_int
    lib.fa_qcache_evict.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, vp, i64, vp, vp] + [i64] * 6 + [vp]
    lib.fa_qcache_evict.restype = ctypes.c_int
    lib.fa_check_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.fa_check_device_status.restype = ctypes.c_int
    lib.fa_get_device_status.argtypes = [vp]
    lib.fa_get_device_status.restype = ctypes.c_int
    lib.fa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.fa_set_wait_limit_ns.restype = ctypes.c_int
    lib.fa_debug_skip_k_tile.argtypes = [ctypes.c_int]
    lib.fa_debug_skip_k_tile.restype = ctypes.c_int
    lib.fa_debug_set_schedule.argtypes = [ctypes.c_int]
    lib.fa_debug_set_schedule.restype = ctypes.c_int
    lib.fa_debug_decode_plan.argtypes = [i64, i64, i64, i64, i64, i64, ctypes.POINTER(ctypes.c_int),
                                         ctypes.POINTER(ctypes.c_int)]
    lib.fa_debug_decode_plan.restype = ctypes.c_int
    lib.fa_status_string.argtypes = [ctypes.c_int]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = ctypes.c_int
    _lib = lib
    return lib


def version() -> int:
    return int(library().fa_version())


def _stream_handle(stream, device: int | None = None):
    """The raw cudaStream_t of ``stream`` as an int, else the current stream
    of ``device`` (default: the current device)."""
    import torch

    if stream is not None:
        return int(stream.cuda_stream)
    if device is None:
        device = torch.cuda.current_device()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return int(raw(device))
    return int(torch.cuda.current_stream(device).cuda_stream)


def _stream_on(stream, dev: int) -> None:
    """A stream of another device is refused: the handle of that device's default
    stream is 0, which would mean the current device's."""
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device} but the tensors are on cuda:{dev}")


def _under(stream, t):
    """The context of a call on tensor t whose results belong to ``stream``."""
    import torch

    if t.is_cuda:
        _stream_on(stream, t.get_device())
    return torch.cuda.stream(stream)


def _on_current_device(dev: int) -> None:
    """The C entry points launch on the calling thread's current device, so
    the tensors must live there."""
    import torch

    cur = torch.cuda.current_device()
    if dev != cur:
        raise ValueError(f"tensors are on cuda:{dev} but the current device is cuda:{cur}: "
                         f"call under torch.cuda.device({dev})")


def _cuda_device() -> int:
    """The current CUDA device of this thread (torch.cuda.current_device without
    its initialisation check: a CUDA tensor is at hand)."""
    import torch

    get = getattr(torch._C, "_cuda_getDevice", None)
    return get() if get is not None else torch.cuda.current_device()


def _fast_ok(dev: int, shape, dtype, *ts) -> bool:
    """One pass over tensors that must all be contiguous, of this dtype and
    shape, on CUDA device dev (the common case; any failure is reported by
    the detailed checks)."""
    for t in ts:
        if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            return False
    return True


def _check(q, k, v):
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bf16, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dim() != 4:
            raise ValueError(f"{name} must be (B, H, N, d), got shape {tuple(t.shape)}")
    if not (q.shape == k.shape == v.shape):
        raise ValueError(f"q, k, v shapes differ: {tuple(q.shape)} {tuple(k.shape)} {tuple(v.shape)}")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")


def _check_out(name, t, shape, dtype, device):
    """An output tensor the kernels write: CUDA, contiguous, of exactly this
    shape and dtype, on the inputs' device."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def fwd_into(q, k, v, o, lse, causal: bool = False, scale: float | None = None, stream=None):
    """Runs the kernel into caller-provided ``o`` (bf16, the shape of q) and
    ``lse`` (fp32, (B, H, N))."""
    import torch

    shape = q.shape
    dev = q.get_device()
    if not (dev >= 0 and len(shape) == 4 and _fast_ok(dev, shape, torch.bfloat16, q, k, v, o)
            and lse.get_device() == dev and lse.dtype is torch.float32 and lse.shape == shape[:3]
            and lse.is_contiguous()):
        _check(q, k, v)
        _check_out("o", o, q.shape, torch.bfloat16, q.device)
        _check_out("lse", lse, tuple(q.shape[:3]), torch.float32, q.device)
    _on_current_device(dev)
    B, H, N, d = shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rc = library().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                          1 if causal else 0, float(scale), _stream_handle(stream, dev))
    if rc != 0:
        raise FaError(rc, "fa_fwd")
    return o, lse


def fwd(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """Attention forward; returns ``(o, lse)`` (see module docstring)."""
    import torch

    _check(q, k, v)
    B, H, N, d = (int(s) for s in q.shape)
    with torch.cuda.device(q.device):
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        return fwd_into(q, k, v, o, lse, causal, scale, stream)


def bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    """Workspace bytes fa_bwd needs for these sizes."""
    out = ctypes.c_size_t(0)
    rc = library().fa_bwd_workspace_bytes(int(B), int(H), int(N), int(d), ctypes.byref(out))
    if rc != 0:
        raise FaError(rc, "fa_bwd_workspace_bytes")
    return int(out.value)


def bwd_into(q, k, v, o, lse, do, dq, dk, dv, workspace, causal: bool = False, scale: float | None = None,
             stream=None):
    """Backward into caller-provided dq, dk, dv (bf16) and workspace (a CUDA
    tensor of at least bwd_workspace_bytes bytes)."""
    import torch

    _check(q, k, v)
    _check(o, do, dq)
    _check(dk, dv, dq)
    if not (q.shape == o.shape == do.shape == dq.shape):
        raise ValueError("o, do, dq, dk, dv must have the shape of q")
    B, H, N, d = (int(s) for s in q.shape)
    if not (q.device == o.device == do.device == dq.device == dk.device == dv.device):
        raise ValueError("q, k, v, o, do, dq, dk, dv must be on one device")
    _check_out("lse", lse, (B, H, N), torch.float32, q.device)
    if not workspace.is_cuda or workspace.device != q.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    ws_bytes = workspace.numel() * workspace.element_size()
    dev = q.get_device()
    _on_current_device(dev)
    vp = ctypes.c_void_p
    rc = library().fa_bwd(vp(q.data_ptr()), vp(k.data_ptr()), vp(v.data_ptr()), vp(o.data_ptr()),
                          vp(lse.data_ptr()), vp(do.data_ptr()), vp(dq.data_ptr()), vp(dk.data_ptr()),
                          vp(dv.data_ptr()), B, H, N, d, int(bool(causal)), float(scale), vp(workspace.data_ptr()),
                          ws_bytes, _stream_handle(stream, dev))
    if rc != 0:
        raise FaError(rc, "fa_bwd")
    return dq, dk, dv


def bwd(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None, stream=None):
    """Gradients ``(dq, dk, dv)`` of the attention forward (o, lse from
    :func:`fwd` with the same causal and scale) for the output gradient do."""
    import torch

    _check(q, k, v)
    B, H, N, d = (int(s) for s in q.shape)
    with torch.cuda.device(q.device):
        ws = torch.empty(bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        return bwd_into(q, k, v, o, lse, do, dq, dk, dv, ws, causal, scale, stream)


def bias_gelu_dropout(x, bias, keep=None, p: float = 0.0, out=None, stream=None):
    """y = dropout(gelu(x + bias)) for x (rows, cols) bf16 and bias (cols,) bf16
    on the GPU; keep: int32/uint32 CUDA tensor of ceil(rows*cols/32) words of
    keep bits (bit e % 32 of word e // 32 keeps flat element e), or None to
    keep all; kept values are scaled by 1/(1-p).  Returns y (bf16, like x)."""
    import torch

    for name, t in (("x", x), ("bias", bias)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor")
    if x.dim() != 2 or bias.shape != (x.shape[1],):
        raise ValueError(f"x (rows, cols) and bias (cols,) expected: {tuple(x.shape)} {tuple(bias.shape)}")
    rows, cols = (int(s) for s in x.shape)
    if keep is not None:
        if not keep.is_cuda or keep.dtype not in (torch.int32, torch.uint32) or not keep.is_contiguous():
            raise ValueError("keep must be a contiguous CUDA int32/uint32 tensor of mask words")
        if keep.numel() * 32 < rows * cols:
            raise ValueError("keep holds fewer bits than x has elements")
    if (keep is not None and keep.device != x.device) or bias.device != x.device:
        raise ValueError("x, bias and keep must be on one device")
    if out is not None:
        _check_out("out", out, x.shape, torch.bfloat16, x.device)
    dev = x.get_device()
    _on_current_device(dev)
    y = torch.empty_like(x) if out is None else out
    vp = ctypes.c_void_p
    rc = library().fa_bias_gelu_dropout(vp(x.data_ptr()), vp(bias.data_ptr()),
                                        vp(keep.data_ptr() if keep is not None else 0), vp(y.data_ptr()), rows,
                                        cols, float(p), _stream_handle(stream, dev))
    if rc != 0:
        raise FaError(rc, "fa_bias_gelu_dropout")
    return y


def _check_decode(q, k, v):
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous CUDA bf16 (B, H, N, d) tensor")
    if k.shape != v.shape or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError(f"q (B, H, Nq, d) and k, v (B, H, Nk, d) expected: {tuple(q.shape)} {tuple(k.shape)}")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")


def decode_workspace_bytes(B: int, H: int, Nq: int, Nk: int, d: int, causal: bool = False) -> int:
    """Workspace bytes fa_decode needs for these sizes on the current device."""
    out = ctypes.c_size_t(0)
    rc = library().fa_decode_workspace_bytes(int(B), int(H), int(Nq), int(Nk), int(d), int(bool(causal)),
                                             ctypes.byref(out))
    if rc != 0:
        raise FaError(rc, "fa_decode_workspace_bytes")
    return int(out.value)


def decode_into(q, k, v, o, lse, workspace, causal: bool = False, scale: float | None = None, stream=None):
    """Decode attention into caller-provided o (bf16, the shape of q), lse
    (fp32, (B, H, Nq)) and workspace (a CUDA tensor of at least
    decode_workspace_bytes bytes, or None when that is 0)."""
    import torch

    _check_decode(q, k, v)
    B, H, Nq, d = (int(s) for s in q.shape)
    Nk = int(k.shape[2])
    _check_out("o", o, q.shape, torch.bfloat16, q.device)
    _check_out("lse", lse, (B, H, Nq), torch.float32, q.device)
    if workspace is not None and (not workspace.is_cuda or workspace.device != q.device
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dev = q.get_device()
    _on_current_device(dev)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p(0)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = library().fa_decode(ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
                             ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(o.data_ptr()),
                             ctypes.c_void_p(lse.data_ptr()), B, H, Nq, Nk, d, int(bool(causal)), float(scale),
                             ws_ptr, ws_bytes, _stream_handle(stream, dev))
    if rc != 0:
        raise FaError(rc, "fa_decode")
    return o, lse


def decode(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """Attention of q (B, H, Nq, d), Nq <= 8, against the cache k, v
    (B, H, Nk, d); query i stands at key position Nk - Nq + i.  Returns
    ``(o (B, H, Nq, d) bf16, lse (B, H, Nq) fp32)``."""
    import torch

    _check_decode(q, k, v)
    B, H, Nq, d = (int(s) for s in q.shape)
    with torch.cuda.device(q.device):
        nbytes = decode_workspace_bytes(B, H, Nq, int(k.shape[2]), d, causal)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        o = torch.empty_like(q)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        return decode_into(q, k, v, o, lse, ws, causal, scale, stream)


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: int = 0, slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """The frequencies of rotary positions over ``rot`` channels, for
    :func:`rope`: an int64 tensor (rot/2) of turns per position in units of
    2^-64 of a turn, and the factor that scales the turned channels.

    Pair i turns base ** (-2 i / rot) radians a position.  ``scaling`` stretches
    that to contexts ``factor`` times as long: "linear" divides every frequency
    by it; "base" raises the base so that the slowest pair is divided by it and
    the fastest kept; "parts" divides the pairs that make fewer than ``slow``
    turns over ``original_length`` positions, keeps those that make more than
    ``fast``, blends linearly between, and scales the channels by
    0.1 ln(factor) + 1.  Computed in 64-bit floating point: a frequency is good to
    2^-46 of itself, so an angle at position t to 2^-46 of the turns made by then."""
    import torch

    if rot < 2 or rot % 2 or not (math.isfinite(base) and base > 1.0):
        raise ValueError("rot must be even and at least 2, base above 1")
    if scaling not in ("none", "linear", "base", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling != "none" and not (math.isfinite(factor) and factor >= 1.0):
        raise ValueError("factor must be at least 1")
    if scaling == "parts" and not (original_length > 0 and 0 < slow < fast):
        raise ValueError("parts needs original_length > 0 and 0 < slow < fast")
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0
    words = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot) / (2.0 * math.pi)  # turns a position
        if scaling == "linear":
            f /= factor
        elif scaling == "parts":
            keep = min(1.0, max(0.0, (original_length * f - slow) / (fast - slow)))
            f = f * keep + f / factor * (1.0 - keep)
        u = int(round(f * 2.0 ** 64)) & (2 ** 64 - 1)
        words.append(u - 2 ** 64 if u >= 2 ** 63 else u)
    return torch.tensor(words, dtype=torch.int64, device=device), amplitude


def _check_rows(name, t, dev=None):
    """A bf16 CUDA tensor (B, H, N, d) whose channels adjoin."""
    import torch

    if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4:
        raise ValueError(f"{name} must be a CUDA bf16 (B, H, N, d) tensor")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name}'s channels must adjoin (last stride 1)")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")


def _strides(t):
    """A host array of the batch, head and position strides, or None when contiguous."""
    if t.is_contiguous():
        return None
    return (ctypes.c_int64 * 3)(t.stride(0), t.stride(1), t.stride(2))


def _check_int32(name, t, shape, dev):
    import torch

    if t.get_device() != dev or t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor on cuda:{dev}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_rope(q, k, freqs, positions, lens, layout):
    """Checks of everything but the results; returns (device, B, H, Hk, N, d)."""
    import torch

    if layout != "half" and layout != "interleaved":
        raise ValueError(f"unknown layout {layout!r}")
    _check_rows("q", q)
    dev = q.get_device()
    B, H, N, d = q.shape
    Hk = 0
    if k is not None:
        _check_rows("k", k, dev)
        Bk, Hk, Nk, dk = k.shape
        if Bk != B or Nk != N or dk != d:
            raise ValueError(f"k must be (B, Hk, N, d) like q: {tuple(q.shape)} {tuple(k.shape)}")
    if freqs.get_device() != dev or freqs.dtype is not torch.int64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous CUDA int64 vector (see rope_frequencies)")
    if positions is not None:
        if positions.get_device() != dev or positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("positions must be a CUDA int32 or int64 tensor")
        if tuple(positions.shape) not in ((N,), (B, N)) or (N > 1 and positions.stride(-1) != 1):
            raise ValueError("positions must be (N,) or (B, N), the positions of a sequence adjoining")
    if lens is not None:
        _check_int32("lens", lens, (B,), dev)
    return dev, B, H, Hk, N, d


def _rope_call(q, k, q_out, k_out, freqs, positions, lens, layout, factor, inverse, stream, sizes):
    dev, B, H, Hk, N, d = sizes
    pos_ptr, pos_bytes, pos_stride = 0, 0, 0
    if positions is not None:
        pos_ptr, pos_bytes = positions.data_ptr(), positions.element_size()
        pos_stride = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    if k is None:
        kp, ks, kop, kos = 0, None, 0, None
    else:
        kp, ks, kop, kos = k.data_ptr(), _strides(k), k_out.data_ptr(), _strides(k_out)
    rc = library().fa_rope(q.data_ptr(), _strides(q), kp, ks, q_out.data_ptr(), _strides(q_out), kop, kos, B, H, Hk, N,
                           d, freqs.data_ptr(), 2 * freqs.numel(), layout == "interleaved", float(factor), bool(inverse),
                           pos_ptr, pos_bytes, pos_stride, 0 if lens is None else lens.data_ptr(),
                           _stream_handle(stream, dev))
    if rc != 0:
        raise FaError(rc, "fa_rope")
    return q_out, k_out


def rope_into(q, k, q_out, k_out, freqs, positions=None, lens=None, layout: str = "half", factor: float = 1.0,
              inverse: bool = False, stream=None):
    """:func:`rope` into caller-provided tensors of q's and k's shapes (each
    may be its own input; strided views are fine)."""
    sizes = _check_rope(q, k, freqs, positions, lens, layout)
    dev = sizes[0]
    _check_rows("q_out", q_out, dev)
    if q_out.shape != q.shape:
        raise ValueError("q_out must have the shape of q")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    if k is not None:
        _check_rows("k_out", k_out, dev)
        if k_out.shape != k.shape:
            raise ValueError("k_out must have the shape of k")
    _on_current_device(dev)
    _stream_on(stream, dev)
    return _rope_call(q, k, q_out, k_out, freqs, positions, lens, layout, factor, inverse, stream, sizes)


def rope(q, k, freqs, positions=None, lens=None, layout: str = "half", factor: float = 1.0, inverse: bool = False,
         stream=None):
    """Turns q (B, H, N, d) and k (B, Hk, N, d; or None) by their positions and
    returns new contiguous tensors.  freqs and factor: :func:`rope_frequencies`;
    2 * len(freqs) channels are turned, the others copied.  positions: int32 or
    int64 (N,) or (B, N); or lens, int32 (B,): row i stands at lens[b] - N + i
    (a cache's lens only as long as nothing was evicted from it: kept keys stand
    where they were produced); or neither: row i stands at i.  Strided views (heads of a fused
    projection) are taken as they are."""
    import torch

    if stream is not None:  # the results belong to the stream that writes them
        with _under(stream, q):
            return rope(q, k, freqs, positions, lens, layout, factor, inverse)
    sizes = _check_rope(q, k, freqs, positions, lens, layout)
    dev = sizes[0]
    if _cuda_device() != dev:
        with torch.cuda.device(dev):
            return rope(q, k, freqs, positions, lens, layout, factor, inverse)
    q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    k_out = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
    return _rope_call(q, k, q_out, k_out, freqs, positions, lens, layout, factor, inverse, None, sizes)


def rope_bwd(dq, dk, freqs, positions=None, lens=None, layout: str = "half", factor: float = 1.0, stream=None):
    """The gradient of :func:`rope`: dLoss/dq and dLoss/dk from the gradients of
    its results (the transposed map; the other arguments as in the forward)."""
    return rope(dq, dk, freqs, positions, lens, layout, factor, True, stream)


QCACHE_PAGE = 64


def qcache_pool(num_pages: int, Hkv: int, d: int, device="cuda"):
    """An empty pool for a 4-bit cache: uint8 (num_pages, Hkv, 72 * D), D = 64
    for d <= 64, else 128.  A page holds 64 keys of every kv head; its
    contents need not start at anything."""
    import torch

    if num_pages < 1 or Hkv < 1 or d < 8 or d > 128 or d % 8:
        raise ValueError("num_pages and Hkv must be positive, d a multiple of 8 up to 128")
    return torch.empty((num_pages, Hkv, 72 * (64 if d <= 64 else 128)), dtype=torch.uint8, device=device)


def _check_qcache(pool, table, lens, d):
    """The cache's tensors; returns (device, B, num_pages, Hkv, max_pages)."""
    import torch

    dev = pool.get_device()
    if dev < 0 or pool.dtype is not torch.uint8 or pool.dim() != 3 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous CUDA uint8 (pages, Hkv, bytes) tensor (see qcache_pool)")
    num_pages, Hkv, block = pool.shape
    if d is not None and block != (4608 if d <= 64 else 9216):
        raise ValueError(f"pool was made for another head size than {d}")
    if block != 4608 and block != 9216:
        raise ValueError("pool's blocks must hold 72 * 64 or 72 * 128 bytes")
    if table.dim() != 2:
        raise ValueError("table must be (B, max_pages)")
    _check_int32("table", table, None, dev)
    B, max_pages = table.shape
    _check_int32("lens", lens, (B,), dev)
    return dev, B, num_pages, Hkv, max_pages


def qcache_append(k, v, pool, table, lens, k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Rounds k and v (B, Hkv, N, d) into the cache as the newest N keys of each
    sequence: row i becomes key lens[b] - N + i (rows of negative position are
    padding).  lens counts the new keys already."""
    _check_rows("k", k)
    B, Hkv, N, d = k.shape
    dev, Bc, num_pages, Hp, max_pages = _check_qcache(pool, table, lens, d)
    _check_rows("v", v, dev)
    if v.shape != k.shape or Bc != B or Hp != Hkv or k.get_device() != dev:
        raise ValueError(f"k and v must be (B, Hkv, N, d) of the cache's batch, heads and device: {tuple(k.shape)} "
                         f"{tuple(v.shape)}")
    _on_current_device(dev)
    _stream_on(stream, dev)
    rc = library().fa_qcache_append(k.data_ptr(), _strides(k), v.data_ptr(), _strides(v), B, Hkv, N, d,
                                    float(k_scale), float(v_scale), pool.data_ptr(), num_pages, table.data_ptr(), max_pages, lens.data_ptr(),
                                    _stream_handle(stream, dev))
    if rc != 0:
        raise FaError(rc, "fa_qcache_append")


def qcache_read(pool, table, lens, n: int, d: int, newest: bool = False, k_scale: float = 1.0, v_scale: float = 1.0,
                stream=None):
    """Keys 0 .. n-1 (or the newest n) of every sequence as bf16 tensors k and v
    (B, Hkv, n, d); rows where no key is are zero."""
    import torch

    if stream is not None:
        with _under(stream, pool):
            return qcache_read(pool, table, lens, n, d, newest, k_scale, v_scale)
    dev, B, num_pages, Hkv, max_pages = _check_qcache(pool, table, lens, d)
    n = int(n)
    if n < 1:
        raise ValueError("n must be positive")
    if _cuda_device() != dev:
        with torch.cuda.device(dev):
            return qcache_read(pool, table, lens, n, d, newest, k_scale, v_scale)
    k = torch.empty((B, Hkv, n, d), dtype=torch.bfloat16, device=pool.device)
    v = torch.empty_like(k)
    rc = library().fa_qcache_read(pool.data_ptr(), num_pages, table.data_ptr(), max_pages, lens.data_ptr(),
                                  k.data_ptr(), v.data_ptr(), B, Hkv, n, d, bool(newest), float(k_scale), float(v_scale),
                                  _stream_handle(None, dev))
    if rc != 0:
        raise FaError(rc, "fa_qcache_read")
    return k, v


def _check_qcache_query(q, pool, table, lens):
    """Checks of a call with queries; returns (device, num_pages, Hkv, max_pages)."""
    import torch

    if not q.is_cuda or q.dtype is not torch.bfloat16 or not q.is_contiguous() or q.dim() != 4:
        raise ValueError("q must be a contiguous CUDA bf16 (B, H, Nq, d) tensor")
    B, H, Nq, d = q.shape
    dev, Bc, num_pages, Hkv, max_pages = _check_qcache(pool, table, lens, d)
    if Bc != B or q.get_device() != dev:
        raise ValueError("q and the cache must have one batch size and be on one device")
    return dev, num_pages, Hkv, max_pages


def qcache_decode_workspace_bytes(B: int, H: int, Hkv: int, Nq: int, d: int, max_pages: int) -> int:
    """Workspace bytes fa_qcache_decode needs for these sizes on the current device."""
    out = ctypes.c_size_t(0)
    rc = library().fa_qcache_decode_workspace_bytes(int(B), int(H), int(Hkv), int(Nq), int(d), int(max_pages),
                                                    ctypes.byref(out))
    if rc != 0:
        raise FaError(rc, "fa_qcache_decode_workspace_bytes")
    return int(out.value)


@functools.lru_cache(maxsize=256)
def _qcache_workspace(dev, B, H, Hkv, Nq, d, max_pages):
    """The workspace size on device dev (the current one), a function of the sizes alone."""
    return qcache_decode_workspace_bytes(B, H, Hkv, Nq, d, max_pages)


def _qcache_decode_call(q, pool, table, lens, o, lse, workspace, causal, scale, k_scale, v_scale, stream, sizes):
    dev, num_pages, Hkv, max_pages = sizes
    B, H, Nq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rc = library().fa_qcache_decode(q.data_ptr(), pool.data_ptr(), num_pages, table.data_ptr(), max_pages,
                                    lens.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, Hkv, Nq, d, bool(causal),
                                    float(scale), float(k_scale), float(v_scale), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    if rc != 0:
        raise FaError(rc, "fa_qcache_decode")
    return o, lse


def qcache_decode_into(q, pool, table, lens, o, lse, workspace, causal: bool = False, scale: float | None = None,
                       k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """:func:`qcache_decode` into caller-provided o (bf16, like q), lse (fp32,
    (B, H, Nq)) and workspace (a contiguous CUDA tensor of at least
    qcache_decode_workspace_bytes bytes)."""
    import torch

    sizes = _check_qcache_query(q, pool, table, lens)
    dev = sizes[0]
    _check_out("o", o, q.shape, torch.bfloat16, q.device)
    _check_out("lse", lse, q.shape[:3], torch.float32, q.device)
    if not workspace.is_cuda or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    _on_current_device(dev)
    _stream_on(stream, dev)
    return _qcache_decode_call(q, pool, table, lens, o, lse, workspace, causal, scale, k_scale, v_scale, stream, sizes)


def qcache_decode(q, pool, table, lens, causal: bool = False, scale: float | None = None, k_scale: float = 1.0,
                  v_scale: float = 1.0, stream=None):
    """Attention of q (B, H, Nq, d), Nq <= 8, against the 4-bit cache: query head
    h reads kv head h // (H // Hkv), query i sees the keys of its sequence (up
    to key lens[b] - Nq + i when causal).  Returns ``(o (B, H, Nq, d) bf16, lse
    (B, H, Nq) fp32)``; a query that sees no key gives 0 and -inf."""
    import torch

    if stream is not None:  # the workspace and the results belong to the stream that writes them
        with _under(stream, q):
            return qcache_decode(q, pool, table, lens, causal, scale, k_scale, v_scale)
    sizes = _check_qcache_query(q, pool, table, lens)
    dev, _, Hkv, max_pages = sizes
    if _cuda_device() != dev:
        with torch.cuda.device(dev):
            return qcache_decode(q, pool, table, lens, causal, scale, k_scale, v_scale)
    B, H, Nq, d = q.shape
    on = q.device
    ws = torch.empty(_qcache_workspace(dev, B, H, Hkv, Nq, d, max_pages), dtype=torch.uint8, device=on)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=on)
    return _qcache_decode_call(q, pool, table, lens, o, lse, ws, causal, scale, k_scale, v_scale, None, sizes)


def qcache_weights(q, lse, pool, table, lens, weights, causal: bool = False, scale: float | None = None,
                   k_scale: float = 1.0, out=None, stream=None):
    """weights (B, Hkv, W) fp32 plus the attention weight that q's rows give each
    cached key: exp(scale q.k - lse) summed over the query rows of the key's kv
    head, with q, causal and scale as in the decode call that returned lse.
    ``out`` may be weights itself."""
    import torch

    if stream is not None:
        with _under(stream, q):
            return qcache_weights(q, lse, pool, table, lens, weights, causal, scale, k_scale, out)
    dev, num_pages, Hkv, max_pages = _check_qcache_query(q, pool, table, lens)
    if _cuda_device() != dev:
        with torch.cuda.device(dev):
            return qcache_weights(q, lse, pool, table, lens, weights, causal, scale, k_scale, out)
    B, H, Nq, d = q.shape
    if not _fast_ok(dev, (B, H, Nq), torch.float32, lse):
        _check_out("lse", lse, (B, H, Nq), torch.float32, q.device)
    if weights.dim() != 3:
        raise ValueError("weights must be (B, Hkv, W)")
    if not _fast_ok(dev, (B, Hkv, weights.shape[2]), torch.float32, weights):
        _check_out("weights", weights, (B, Hkv, weights.shape[2]), torch.float32, q.device)
    if out is not None:
        _check_out("out", out, weights.shape, torch.float32, q.device)
    else:
        out = torch.empty_like(weights)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rc = library().fa_qcache_weights(q.data_ptr(), lse.data_ptr(), pool.data_ptr(), num_pages, table.data_ptr(),
                                     max_pages, lens.data_ptr(), weights.data_ptr(), out.data_ptr(),
                                     weights.shape[2], B, H, Hkv, Nq, d, bool(causal), float(scale),
                                     float(k_scale), _stream_handle(None, dev))
    if rc != 0:
        raise FaError(rc, "fa_qcache_weights")
    return out


def qcache_evict(pool, table, lens, weights, keep: int, sink: int = 0, recent: int = 0, table_out=None, stream=None):
    """Cuts every sequence back to its ``keep`` keys: the first ``sink``, the last
    ``recent`` and the heaviest between (a choice per kv head; of equal weights
    the lowest positions).  The kept keys move, in order, to the pages of
    table_out, or within the sequence's own pages when it is None.  Returns
    ``(kept, lens, weights)``: the kept keys' former positions, int32 (B, Hkv,
    keep), -1 after the last; the new lengths; the kept keys' weights at their
    new places, 0 after them (like weights)."""
    import torch

    if stream is not None:
        with _under(stream, pool):
            return qcache_evict(pool, table, lens, weights, keep, sink, recent, table_out)
    dev, B, num_pages, Hkv, max_pages = _check_qcache(pool, table, lens, None)
    if _cuda_device() != dev:
        with torch.cuda.device(dev):
            return qcache_evict(pool, table, lens, weights, keep, sink, recent, table_out)
    if weights.dim() != 3:
        raise ValueError("weights must be (B, Hkv, W)")
    if not _fast_ok(dev, (B, Hkv, weights.shape[2]), torch.float32, weights):
        _check_out("weights", weights, (B, Hkv, weights.shape[2]), torch.float32, pool.device)
    if table_out is None:
        table_out = table
    elif table_out.dim() != 2 or table_out.shape[0] != B:
        raise ValueError("table_out must be (B, max_pages_out)")
    _check_int32("table_out", table_out, None, dev)
    keep, sink, recent = int(keep), int(sink), int(recent)
    if keep < 1 or sink < 0 or recent < 0 or sink + recent > keep:
        raise ValueError("keep must be positive, sink and recent not negative and together at most keep")
    kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device=pool.device)
    lens_out = torch.empty_like(lens)
    weights_out = torch.empty_like(weights)
    rc = library().fa_qcache_evict(pool.data_ptr(), num_pages, table.data_ptr(), max_pages, lens.data_ptr(),
                                   table_out.data_ptr(), table_out.shape[1], weights.data_ptr(),
                                   weights_out.data_ptr(), weights.shape[2], kept.data_ptr(), lens_out.data_ptr(), B,
                                   Hkv, pool.shape[2] // 72, keep, sink, recent, _stream_handle(None, dev))
    if rc != 0:
        raise FaError(rc, "fa_qcache_evict")
    return kept, lens_out, weights_out


def check_device_status(stream=None) -> int:
    """Synchronises the stream and returns the device status (0 = ok, 4 = a wait
    timed out, 1 = a cache call skipped a page or length out of range); raises
    FaError on a CUDA error."""
    where = ctypes.c_uint32(0)
    rc = library().fa_check_device_status(_stream_handle(stream), ctypes.byref(where))
    if rc == 3:
        raise FaError(rc, "fa_check_device_status")
    return rc


def get_device_status(stream=None) -> int:
    """fa_get_device_status: synchronises the stream and returns the device
    status (0 = ok, 4 = a wait timed out, 1 = a cache call skipped a page or
    length out of range); raises FaError on a CUDA error."""
    rc = library().fa_get_device_status(_stream_handle(stream))
    if rc == 3:
        raise FaError(rc, "fa_get_device_status")
    return rc


def set_wait_limit_ns(ns: int) -> None:
    library().fa_set_wait_limit_ns(int(ns))


def debug_skip_k_tile(tile: int) -> None:
    """Test hook: see fa_debug_skip_k_tile in include/fa.h (-1 turns it off)."""
    rc = library().fa_debug_skip_k_tile(int(tile))
    if rc != 0:
        raise FaError(rc, "fa_debug_skip_k_tile")


def debug_set_schedule(order: int) -> None:
    """Test hook: see fa_debug_set_schedule in include/fa.h (-1: the order by
    size, 0: heavy/light pairs, 1: cost order)."""
    rc = library().fa_debug_set_schedule(int(order))
    if rc != 0:
        raise FaError(rc, "fa_debug_set_schedule")


def debug_decode_plan(B: int, H: int, Nq: int, Nk: int, d: int, wave: int) -> tuple[int, int]:
    """Test hook: the (splits, keys per chunk) that fa_decode would use if
    ``wave`` CTAs of its partial kernel were resident at once (host
    arithmetic only; see fa_debug_decode_plan in include/fa.h)."""
    splits, chunk = ctypes.c_int(0), ctypes.c_int(0)
    rc = library().fa_debug_decode_plan(B, H, Nq, Nk, d, wave, ctypes.byref(splits), ctypes.byref(chunk))
    if rc != 0:
        raise FaError(rc, "fa_debug_decode_plan")
    return splits.value, chunk.value
