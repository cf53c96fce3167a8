"""Thin Python binding over ``libra.so``.  The functions carry the C ABI's
names (include/ra.h).  This module only marshals arguments: it takes torch
tensors, passes raw pointers, sizes and the stream, and turns status codes
into exceptions.  Every step of the computation runs in the library's CUDA
kernels.  There is no fallback.  If ``libra.so`` is missing, the first call
raises ``RaError``.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libra.so")
SERVE_PATH = os.path.join(_PKG, "_serve.so")

RA_OK = 0
RA_ERR_INVALID = -1
RA_ERR_UNSUPPORTED = -2
RA_ERR_CUDA = -3
RA_ERR_TIMEOUT = -4
RA_ERR_ALLOC = -5
RA_F32 = 0
RA_BF16 = 1
LAYOUTS = {"contiguous": 0, "zigzag": 1, "striped": 2}
ABI_VERSION = 3
KERNEL_KINDS = {
    "state_init": 0,
    "block_update_bf16": 1,
    "block_update_f32": 2,
    "merge": 3,
    "finalize": 4,
    "decode_split": 5,
    "decode_combine": 6,
    "bwd_pre": 7,
    "bwd_dq": 8,
    "bwd_dkdv": 9,
    "ring_fused_bf16": 10,
    "ring_fused_f32": 11,
    "paged_extend": 12,
    "paged_release": 13,
    "qk_norm_rope": 14,
    "qk_norm_rope_bwd": 15,
    "qk_norm_weight_grad": 16,
    "paged_append": 17,
    "paged_decode": 18,
    "paged_combine": 19,
}

_lock = threading.Lock()
_lib = None


class RaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [{status}]")
        self.status = status


_SIGNATURES = {
    # name: (argtypes, restype)
    "ra_state_init": ("PPPLiiP", "i"),
    "ra_block_update": ("PPPPPPLiiiLLiiP", "i"),
    "ra_merge": ("PPPPPPLiiP", "i"),
    "ra_finalize": ("PPPPPLiiP", "i"),
    "ra_ring_step": ("PPPPPPLiiiiiiiP", "i"),
    "ra_ring_forward": ("PPPPPLiiiiiiP", "i"),
    "ra_ring_forward_host": ("PPPPPLiiiiiiP", "i"),
    "ra_ring_forward_noalloc": ("PPPPPLiiiiiiP", "i"),
    "ra_block_update_masked": ("PPPPPPLLiiiiiiiLLiLLPiiP", "i"),
    "ra_ring_step_masked": ("PPPPPPLiiiiLLPiiiiiP", "i"),
    "ra_ring_forward_masked": ("PPPPPLiiiLLPiiiiiP", "i"),
    "ra_decode_partial": ("PPPPPPLLiiiLLiLiP", "i"),
    "ra_ring_backward": ("PPPPPPPPPLiiiiiiP", "i"),
    "ra_ring_backward_masked": ("PPPPPPPPPLiiiLLPiiiiiP", "i"),
    "ra_decode_forward": ("PPPPPLLiLiLiiiiP", "i"),
    "ra_qk_norm_rope": ("PPPPLiiiLLPiiiiPfPPifiP", "i"),
    "ra_qk_norm_rope_backward": ("PPPPPPPPLiiiLLLLPiiiiPfPPifiP", "i"),
    "ra_paged_extend": ("PPiPiPiPiLPPPPPPP", "i"),
    "ra_paged_release": ("PPiPiPiPiPPP", "i"),
    "ra_paged_append": ("PPPPPPLiiiLLLiiLLPPiiPfPPifiP", "i"),
    "ra_paged_decode": ("PPPPPLiiPPiPiiLLLiiiiiP", "i"),
    "ra_device_status": ("P", "i"),
    "ra_selftest_wait_timeout": ("LP", "i"),
    "ra_cached_memory": ("P", "i"),
    "ra_release_cached_memory": ("", "i"),
    "ra_trace_enable": ("i", "i"),
    "ra_trace_reset": ("", "i"),
    "ra_trace_query": ("iPP", "i"),
    "ra_status_string": ("i", "s"),
    "ra_last_error": ("", "s"),
    "ra_abi_version": ("", "i"),
}
_CT = {"P": ctypes.c_void_p, "L": ctypes.c_longlong, "i": ctypes.c_int, "f": ctypes.c_float,
       "s": ctypes.c_char_p}


def lib():
    """Load libra.so once.  Raise RaError if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RaError(RA_ERR_UNSUPPORTED,
                              f"{LIB_PATH} is not built; run __graft_entry__.build() "
                              "(nvcc, sm_103a)")
            L = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in _SIGNATURES.items():
                f = getattr(L, name)
                f.argtypes = [_CT[c] for c in args]
                f.restype = _CT[res]
            if L.ra_abi_version() != ABI_VERSION:
                raise RaError(RA_ERR_UNSUPPORTED, "libra.so ABI version mismatch; rebuild it")
            _lib = L
    return _lib


def _check(rc: int):
    if rc != RA_OK:
        L = lib()
        raise RaError(rc, f"{L.ra_status_string(rc).decode()}: {L.ra_last_error().decode()}")


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# stream= takes a torch.cuda.Stream or a cudaStream_t as an integer.  Ordering
# the streams stays with the caller, and so does keeping the inputs, and the
# outputs that are passed in, until the call's work is done.


def _new(shape, device, stream) -> torch.Tensor:
    """An fp32 output that the caller left out.  Its memory belongs to the
    stream of the call (work on another stream does not hold it, and dropped
    it goes back in that stream's order); the current stream, which may read
    it too, is recorded as its user."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=torch.float32, device=device)
    current, handle = torch.cuda.current_stream(device), _stream(stream)
    if handle == current.cuda_stream:
        return torch.empty(shape, dtype=torch.float32, device=device)
    # (The legacy default stream goes by two handles, of which torch knows one.)
    other = (torch.cuda.default_stream(device) if handle in (0, 1)
             else torch.cuda.ExternalStream(handle, device=device))
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=torch.float32, device=device)
    t.record_stream(current)
    return t


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (token-major)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _qkv_dtype(q: torch.Tensor) -> int:
    if q.dtype == torch.bfloat16:
        return RA_BF16
    if q.dtype == torch.float32:
        return RA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {q.dtype}")


def _shapes(q, k, v):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be [rows, heads, d] (token-major)")
    if k.shape != v.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k and v must match in shape, and q, k, v in dtype")
    if q.shape[2] != k.shape[2]:
        raise ValueError("q and k must share the head dim")
    return q.shape[0], q.shape[1], k.shape[1], q.shape[2]


def _state_shapes(m, l, o, rows, heads, d):
    for name, t, shp in (("m", m, (rows, heads)), ("l", l, (rows, heads)),
                         ("o", o, (rows, heads, d))):
        if tuple(t.shape) != shp:
            raise ValueError(f"{name} must have shape {shp}, got {tuple(t.shape)}")


def ra_state_init(m, l, o, stream=None):
    rows, heads, d = o.shape
    _state_shapes(m, l, o, rows, heads, d)
    _check(lib().ra_state_init(_dev(m, "m", torch.float32), _dev(l, "l", torch.float32),
                               _dev(o, "o", torch.float32), rows, d, heads, _stream(stream)))


def ra_block_update(q, k, v, m, l, o, *, q_off: int = 0, kv_off: int = 0, causal: bool = False,
                    stream=None):
    c, heads, kv_heads, d = _shapes(q, k, v)
    if k.shape[0] != c:
        raise ValueError("the query block and the K/V block must have the same length c")
    _state_shapes(m, l, o, c, heads, d)
    _check(lib().ra_block_update(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(m, "m", torch.float32),
        _dev(l, "l", torch.float32), _dev(o, "o", torch.float32), c, d, heads, kv_heads,
        int(q_off), int(kv_off), int(bool(causal)), _qkv_dtype(q), _stream(stream)))


def ra_merge(m_a, l_a, o_a, m_b, l_b, o_b, stream=None):
    rows, heads, d = o_a.shape
    _state_shapes(m_a, l_a, o_a, rows, heads, d)
    _state_shapes(m_b, l_b, o_b, rows, heads, d)
    _check(lib().ra_merge(_dev(m_a, "m_a", torch.float32), _dev(l_a, "l_a", torch.float32),
                          _dev(o_a, "o_a", torch.float32), _dev(m_b, "m_b", torch.float32),
                          _dev(l_b, "l_b", torch.float32), _dev(o_b, "o_b", torch.float32),
                          rows, d, heads, _stream(stream)))


def ra_finalize(m, l, o, out=None, lse=None, stream=None):
    rows, heads, d = o.shape
    _state_shapes(m, l, o, rows, heads, d)
    if out is None:
        out = _new(o.shape, o.device, stream)
    if lse is None:
        lse = _new(m.shape, m.device, stream)
    _state_shapes(lse, lse, out, rows, heads, d)
    _check(lib().ra_finalize(_dev(m, "m", torch.float32), _dev(l, "l", torch.float32),
                             _dev(o, "o", torch.float32), _dev(out, "out", torch.float32),
                             _dev(lse, "lse", torch.float32), rows, d, heads, _stream(stream)))
    return out, lse


def ra_ring_step(q, k, v, m, l, o, *, P: int, s: int, causal: bool, stream=None):
    N, heads, kv_heads, d = _shapes(q, k, v)
    if k.shape[0] != N:
        raise ValueError("q, k and v must cover the same N tokens")
    _state_shapes(m, l, o, N, heads, d)
    _check(lib().ra_ring_step(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(m, "m", torch.float32),
        _dev(l, "l", torch.float32), _dev(o, "o", torch.float32), N, int(P), int(s),
        int(bool(causal)), d, heads, kv_heads, _qkv_dtype(q), _stream(stream)))


def ra_ring_forward(q, k, v, *, P: int, causal: bool, out=None, lse=None, stream=None):
    """Returns (out [N, heads, d] fp32, lse [N, heads] fp32)."""
    N, heads, kv_heads, d = _shapes(q, k, v)
    if k.shape[0] != N:
        raise ValueError("q, k and v must cover the same N tokens")
    if out is None:
        out = _new((N, heads, d), q.device, stream)
    if lse is None:
        lse = _new((N, heads), q.device, stream)
    _state_shapes(lse, lse, out, N, heads, d)
    _check(lib().ra_ring_forward(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out", torch.float32),
        _dev(lse, "lse", torch.float32), N, int(P), int(bool(causal)), d, heads, kv_heads,
        _qkv_dtype(q), _stream(stream)))
    return out, lse


def _layout(layout) -> int:
    if isinstance(layout, str):
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
        return LAYOUTS[layout]
    return int(layout)


def _docs(cu_seqlens):
    """Device pointer and document count of an int32 cu_seqlens tensor (or None)."""
    if cu_seqlens is None:
        return 0, 0
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be 1-D with ndocs + 1 >= 2 entries")
    return _dev(cu_seqlens, "cu_seqlens", torch.int32), cu_seqlens.numel() - 1


def layout_positions(N: int, P: int, layout="contiguous") -> torch.Tensor:
    """Global sequence position held by each row of a ring tensor of N rows
    under `layout` (int64, CPU).  Host index arithmetic for callers that lay
    their tensors out; x_layout = x[argsort(positions)] is not needed, since
    x_layout[r] = x[positions[r]]."""
    lay = _layout(layout)
    if N % P:
        raise ValueError("N must be a multiple of P")
    c = N // P
    r = torch.arange(c, dtype=torch.int64)
    out = []
    for b in range(P):
        if lay == 0:
            out.append(b * c + r)
        elif lay == 1:
            if c % 2:
                raise ValueError("zigzag needs an even block length N / P")
            h = c // 2
            out.append(torch.where(r < h, b * h + r, (2 * P - 1 - b) * h + (r - h)))
        else:
            out.append(r * P + b)
    return torch.cat(out)


def ra_block_update_masked(q, k, v, m, l, o, *, layout="contiguous", P: int = 1,
                           q_block: int = 0, kv_block: int = 0, q_off: int = 0, kv_off: int = 0,
                           causal: bool = False, window: int = 0, n_valid: int = -1,
                           cu_seqlens=None, stream=None):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or k.shape != v.shape:
        raise ValueError("q: [c_q, heads, d]; k, v: [c_kv, kv_heads, d]")
    if k.dtype != q.dtype or v.dtype != q.dtype or q.shape[2] != k.shape[2]:
        raise ValueError("q, k, v must share dtype and head dim")
    c_q, heads, d = q.shape
    c_kv, kv_heads = k.shape[0], k.shape[1]
    _state_shapes(m, l, o, c_q, heads, d)
    cu_ptr, ndocs = _docs(cu_seqlens)
    _check(lib().ra_block_update_masked(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(m, "m", torch.float32),
        _dev(l, "l", torch.float32), _dev(o, "o", torch.float32), c_q, c_kv, d, heads, kv_heads,
        _layout(layout), int(P), int(q_block), int(kv_block), int(q_off), int(kv_off),
        int(bool(causal)), int(window), int(n_valid), cu_ptr, ndocs, _qkv_dtype(q),
        _stream(stream)))


def ra_ring_step_masked(q, k, v, m, l, o, *, P: int, s: int, layout="contiguous",
                        causal: bool = False, window: int = 0, n_valid: int = -1,
                        cu_seqlens=None, stream=None):
    N, heads, kv_heads, d = _shapes(q, k, v)
    if k.shape[0] != N:
        raise ValueError("q, k and v must cover the same N tokens")
    _state_shapes(m, l, o, N, heads, d)
    cu_ptr, ndocs = _docs(cu_seqlens)
    _check(lib().ra_ring_step_masked(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(m, "m", torch.float32),
        _dev(l, "l", torch.float32), _dev(o, "o", torch.float32), N, int(P), int(s),
        _layout(layout), int(bool(causal)), int(window), int(n_valid), cu_ptr, ndocs, d, heads,
        kv_heads, _qkv_dtype(q), _stream(stream)))


def ra_ring_forward_masked(q, k, v, *, P: int, layout="contiguous", causal: bool = False,
                           window: int = 0, n_valid: int = -1, cu_seqlens=None, out=None,
                           lse=None, stream=None):
    """Returns (out [N, heads, d] fp32, lse [N, heads] fp32), rows in q's order."""
    N, heads, kv_heads, d = _shapes(q, k, v)
    if k.shape[0] != N:
        raise ValueError("q, k and v must cover the same N tokens")
    if out is None:
        out = _new((N, heads, d), q.device, stream)
    if lse is None:
        lse = _new((N, heads), q.device, stream)
    _state_shapes(lse, lse, out, N, heads, d)
    cu_ptr, ndocs = _docs(cu_seqlens)
    _check(lib().ra_ring_forward_masked(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out", torch.float32),
        _dev(lse, "lse", torch.float32), N, int(P), _layout(layout), int(bool(causal)),
        int(window), int(n_valid), cu_ptr, ndocs, d, heads, kv_heads, _qkv_dtype(q),
        _stream(stream)))
    return out, lse


def ra_ring_backward_masked(q, k, v, out, lse, dout, *, P: int, layout="contiguous",
                            causal: bool = False, window: int = 0, n_valid: int = -1,
                            cu_seqlens=None, dq=None, dk=None, dv=None, stream=None):
    """Gradients (dq [N, heads, d], dk, dv [N, kv_heads, d], fp32) of the
    ring forward whose outputs are out, lse, for the upstream gradient dout
    (bf16, like q).  Same layout and mask arguments as the forward."""
    N, heads, kv_heads, d = _shapes(q, k, v)
    if k.shape[0] != N:
        raise ValueError("q, k and v must cover the same N tokens")
    _state_shapes(lse, lse, out, N, heads, d)
    if tuple(dout.shape) != (N, heads, d) or dout.dtype != q.dtype:
        raise ValueError("dout must match q in shape and dtype")
    if dq is None:
        dq = _new((N, heads, d), q.device, stream)
    if dk is None:
        dk = _new((N, kv_heads, d), q.device, stream)
    if dv is None:
        dv = _new((N, kv_heads, d), q.device, stream)
    cu_ptr, ndocs = _docs(cu_seqlens)
    _check(lib().ra_ring_backward_masked(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out", torch.float32),
        _dev(lse, "lse", torch.float32), _dev(dout, "dout"), _dev(dq, "dq", torch.float32),
        _dev(dk, "dk", torch.float32), _dev(dv, "dv", torch.float32), N, int(P),
        _layout(layout), int(bool(causal)), int(window), int(n_valid), cu_ptr, ndocs, d, heads,
        kv_heads, _qkv_dtype(q), _stream(stream)))
    return dq, dk, dv


def ra_ring_backward(q, k, v, out, lse, dout, *, P: int, causal: bool, dq=None, dk=None,
                     dv=None, stream=None):
    """ra_ring_backward_masked with the contiguous layout and no extra mask."""
    N, heads, kv_heads, d = _shapes(q, k, v)
    _state_shapes(lse, lse, out, N, heads, d)
    if tuple(dout.shape) != (N, heads, d) or dout.dtype != q.dtype:
        raise ValueError("dout must match q in shape and dtype")
    if dq is None:
        dq = _new((N, heads, d), q.device, stream)
    if dk is None:
        dk = _new((N, kv_heads, d), q.device, stream)
    if dv is None:
        dv = _new((N, kv_heads, d), q.device, stream)
    _check(lib().ra_ring_backward(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out", torch.float32),
        _dev(lse, "lse", torch.float32), _dev(dout, "dout"), _dev(dq, "dq", torch.float32),
        _dev(dk, "dk", torch.float32), _dev(dv, "dv", torch.float32), N, int(P),
        int(bool(causal)), d, heads, kv_heads, _qkv_dtype(q), _stream(stream)))
    return dq, dk, dv


def _decode_shapes(q, k, v):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or k.shape != v.shape:
        raise ValueError("q: [n_q, heads, d]; k, v: [n_kv, kv_heads, d]")
    if k.dtype != q.dtype or v.dtype != q.dtype or q.shape[2] != k.shape[2]:
        raise ValueError("q, k, v must share dtype and head dim")
    return q.shape[0], q.shape[1], k.shape[0], k.shape[1], q.shape[2]


def ra_decode_partial(q, k, v, m, l, o, *, q_off: int, kv_off: int = 0, causal: bool = True,
                      window: int = 0, stream=None):
    """Fold one K/V shard into the state (m, l, o) of n_q query rows, in place."""
    n_q, heads, n_kv, kv_heads, d = _decode_shapes(q, k, v)
    _state_shapes(m, l, o, n_q, heads, d)
    _check(lib().ra_decode_partial(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(m, "m", torch.float32),
        _dev(l, "l", torch.float32), _dev(o, "o", torch.float32), n_q, n_kv, d, heads, kv_heads,
        int(q_off), int(kv_off), int(bool(causal)), int(window), _qkv_dtype(q), _stream(stream)))


def ra_decode_forward(q, k, v, *, P: int, q_off: int | None = None, causal: bool = True,
                      window: int = 0, out=None, lse=None, stream=None):
    """Decode attention of q [n_q, heads, d] against k, v [n_kv, kv_heads, d]
    held as P shards.  q_off defaults to n_kv - n_q (the new tokens are the
    last ones of the history).  Returns (out [n_q, heads, d], lse [n_q, heads])."""
    n_q, heads, n_kv, kv_heads, d = _decode_shapes(q, k, v)
    if q_off is None:
        q_off = n_kv - n_q
    if out is None:
        out = _new((n_q, heads, d), q.device, stream)
    if lse is None:
        lse = _new((n_q, heads), q.device, stream)
    _state_shapes(lse, lse, out, n_q, heads, d)
    kp = _dev(k, "k") if n_kv else 0
    vp = _dev(v, "v") if n_kv else 0
    _check(lib().ra_decode_forward(
        _dev(q, "q"), kp, vp, _dev(out, "out", torch.float32), _dev(lse, "lse", torch.float32),
        n_q, n_kv, int(P), int(q_off), int(bool(causal)), int(window), d, heads, kv_heads,
        _qkv_dtype(q), _stream(stream)))
    return out, lse


# ------------------------------------------------------------------ rotary positions, pages

# These calls are one or two short kernels each, made once or more per layer
# of a serving step.  Their arguments are marshalled by the extension _serve
# (csrc/serve_binding.cpp): the same checks and the same C ABI calls as the
# functions above, at a few microseconds instead of tens.

_serve = None


def _fast():
    """Load the extension once (after libra.so, which it is linked to)."""
    global _serve
    if _serve is None:
        lib()
        if not os.path.exists(SERVE_PATH):
            raise RaError(RA_ERR_UNSUPPORTED,
                          f"{SERVE_PATH} is not built; run __graft_entry__.build()")
        from . import _serve as m

        m.on_status(_check)
        _serve = m
    return _serve


def rope_freqs(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None,
               factor: float = 1.0, original_length: int = 4096, fast_turns: float = 32.0,
               slow_turns: float = 1.0) -> tuple[torch.Tensor, float]:
    """Rotary frequencies (fp64 [rot_dim / 2], radians per position, CPU) and
    the factor on cos and sin, for a head of rot_dim rotated columns.  Host
    arithmetic for callers; pass the frequencies on through rope_phases.

    scaling None: base^(-2i / rot_dim).  "linear": positions divided by
    `factor`.  "ntk": the base raised by factor^(rot_dim / (rot_dim - 2)).
    "yarn" (Peng et al. 2023): frequencies that make at least fast_turns
    turns over original_length positions stay, those below slow_turns are
    divided by `factor`, with a linear blend in pair index between, and cos
    and sin are multiplied by 0.1 ln(factor) + 1."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim={rot_dim} must be even and positive")
    if factor < 1.0:
        raise ValueError(f"factor={factor} must be >= 1")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    f = float(base) ** (-i / rot_dim)
    if scaling is None:
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim >= 4")
        return (base * factor ** (rot_dim / (rot_dim - 2.0))) ** (-i / rot_dim), 1.0
    if scaling != "yarn":
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")

    def pair(turns):  # pair index that makes `turns` turns over original_length
        return rot_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair(fast_turns)), 0), min(math.ceil(pair(slow_turns)), rot_dim - 1)
    ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def rope_phases(freqs: torch.Tensor) -> torch.Tensor:
    """The table the rotary calls take (int64 [rot_dim / 2], on freqs' device)
    from frequencies in radians per position: each as turns per position,
    its fraction in units of 2^-64.  Pass fp64; fp32 values are taken as
    they are."""
    if freqs.dim() != 1:
        raise ValueError("freqs must be 1-D")
    turns = freqs.detach().to(torch.float64) / (2 * math.pi)
    turns = turns - torch.floor(turns)
    hi = torch.floor(turns * 2.0 ** 32)
    lo = torch.floor((turns * 2.0 ** 32 - hi) * 2.0 ** 32)
    return (hi.to(torch.int64) << 32) | lo.to(torch.int64)


def ra_qk_norm_rope(q, k, phases, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                    interleaved: bool = False, mscale: float = 1.0, positions=None, P: int = 1,
                    layout="contiguous", q_out=None, k_out=None, stream=None):
    """Per-head RMS norm (where a weight is given) and rotary positions of
    q [T, heads, d] and k [T, kv_heads, d]; returns dense (q_out, k_out) of
    their dtype.  Rows sit at `positions` (int32 [T]), or where `layout` puts
    the rows of a ring tensor of P blocks.  phases: see rope_phases; None
    leaves the columns unturned."""
    return (_serve or _fast()).qk_norm_rope(
        q, k, phases, q_weight, k_weight, eps, interleaved, mscale, positions, P,
        _layout(layout), q_out, k_out, stream)


def ra_qk_norm_rope_backward(q, k, phases, dq_out, dk_out, *, q_weight=None, k_weight=None,
                             eps: float = 1e-6, interleaved: bool = False, mscale: float = 1.0,
                             positions=None, P: int = 1, layout="contiguous", dq=None, dk=None,
                             dq_weight=None, dk_weight=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ra_qk_norm_rope's inputs
    from those of its outputs (fp32, dense, as ra_ring_backward returns
    them).  dq and dk have q's dtype and may be views of a packed gradient;
    the weights' are fp32 [d], None without that weight."""
    return (_serve or _fast()).qk_norm_rope_backward(
        q, k, phases, dq_out, dk_out, q_weight, k_weight, eps, interleaved, mscale, positions, P,
        _layout(layout), dq, dk, dq_weight, dk_weight, stream)


def ra_paged_extend(lengths, new_tokens, block_table, free_pages, free_count, *, page_size: int,
                    tokens: int, lengths_out=None, free_count_out=None, slots=None,
                    positions=None, cu_tokens=None, status=None, stream=None):
    """Hand out pages for a step's new tokens (all on the device, int32 but
    for slots): block_table's rows are extended in place, and the call
    returns (slots int64 [tokens], positions [tokens], cu_tokens [n_req + 1],
    lengths_out [n_req], free_count_out [1], status [3]).  lengths_out and
    free_count_out may be lengths and free_count themselves; outputs that are
    not passed in are views of one allocation, which lives as long as any of
    them.  A nonzero status (pages missing,
    rows too short, tokens beyond `tokens`) means that the step changed
    nothing."""
    return (_serve or _fast()).paged_extend(
        lengths, new_tokens, block_table, free_pages, free_count, page_size, tokens, lengths_out,
        free_count_out, slots, positions, cu_tokens, status, stream)


def ra_paged_release(lengths, finished, block_table, free_pages, free_count, *, page_size: int,
                     lengths_out=None, free_count_out=None, stream=None):
    """Push the pages of the requests with finished != 0 back on the stack
    free_pages (in place) and set their lengths to 0; returns (lengths_out,
    free_count_out), which may be lengths and free_count themselves; where
    neither is passed in, both are views of one allocation."""
    return (_serve or _fast()).paged_release(
        lengths, finished, block_table, free_pages, free_count, page_size, lengths_out,
        free_count_out, stream)


def ra_paged_append(q, k, v, phases, k_cache, v_cache, slots, positions, *, q_weight=None,
                    k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                    mscale: float = 1.0, q_out=None, stream=None):
    """ra_qk_norm_rope on a step's rows (bf16) with k and v written to their
    pages: row t goes to slots[t] (int64; outside the pages: padding, nothing
    is written) at positions[t] (int32).  Returns q_out, dense like q."""
    return (_serve or _fast()).paged_append(
        q, k, v, phases, k_cache, v_cache, slots, positions, q_weight, k_weight, eps,
        interleaved, mscale, q_out, stream)


def ra_paged_decode(q, k_cache, v_cache, block_table, lengths, *, cu_q=None, n_q: int = 0,
                    window: int = 0, out=None, lse=None, stream=None):
    """Attention of each request's newest tokens q [T, heads, d] (bf16) over
    its pages.  T / n_req rows per request, or rows [cu_q[i], cu_q[i + 1]) of
    request i (int32 [n_req + 1]); lengths (int32 [n_req]) include them.
    With cu_q, n_q says how many rows a request should be expected to have
    (0: T / n_req, the padding rows of a fixed-size step included): it picks
    the kernel, not the result.
    Returns (out [T, heads, d], lse [T, heads]), fp32, views of one allocation
    where not passed in (keeping the LSE keeps both: pass `lse` in, or clone
    it); pass a bf16 `out` for that type."""
    return (_serve or _fast()).paged_decode(
        q, k_cache, v_cache, block_table, lengths, cu_q, n_q, window, out, lse, stream)


def ra_ring_forward_noalloc(q, k, v, *, P: int, causal: bool, out=None, lse=None,
                            stream=None):
    """ra_ring_forward with its l scratch in the library's fixed device array
    (N * heads <= 4,194,304).  It calls no allocator inside the library.
    The output tensors, when not passed in, are still created here by torch.
    Calls that overlap on the GPU share that array and race."""
    N, heads, kv_heads, d = _shapes(q, k, v)
    if k.shape[0] != N:
        raise ValueError("q, k and v must cover the same N tokens")
    if out is None:
        out = _new((N, heads, d), q.device, stream)
    if lse is None:
        lse = _new((N, heads), q.device, stream)
    _state_shapes(lse, lse, out, N, heads, d)
    _check(lib().ra_ring_forward_noalloc(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out", torch.float32),
        _dev(lse, "lse", torch.float32), N, int(P), int(bool(causal)), d, heads, kv_heads,
        _qkv_dtype(q), _stream(stream)))
    return out, lse


def ra_ring_forward_host(q, k, v, *, P: int, causal: bool, out=None, lse=None, stream=None):
    """ra_ring_forward on CPU tensors.  Pinned memory makes the copies
    asynchronous DMA.  The call returns when out and lse are on the host."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU tensor")
    N, heads, kv_heads, d = _shapes(q, k, v)
    if out is None:
        out = torch.empty((N, heads, d), dtype=torch.float32, pin_memory=q.is_pinned())
    if lse is None:
        lse = torch.empty((N, heads), dtype=torch.float32, pin_memory=q.is_pinned())
    _check(lib().ra_ring_forward_host(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), N, int(P),
        int(bool(causal)), d, heads, kv_heads, _qkv_dtype(q), _stream(stream)))
    return out, lse


def ra_device_status(stream=None):
    _check(lib().ra_device_status(_stream(stream)))


def ra_selftest_wait_timeout(limit_cycles: int, stream=None) -> int:
    return lib().ra_selftest_wait_timeout(int(limit_cycles), _stream(stream))


def ra_cached_memory() -> int:
    """Bytes the library's scratch pool holds on the current device."""
    n = ctypes.c_longlong(0)
    _check(lib().ra_cached_memory(ctypes.addressof(n)))
    return int(n.value)


def ra_release_cached_memory():
    _check(lib().ra_release_cached_memory())


def ra_trace_enable(on: bool = True):
    _check(lib().ra_trace_enable(int(bool(on))))


def ra_trace_reset():
    _check(lib().ra_trace_reset())


def ra_trace_query(kind) -> tuple[int, float]:
    """Returns (launches, total device ms) of one kernel kind since the last reset."""
    k = KERNEL_KINDS[kind] if isinstance(kind, str) else int(kind)
    n = ctypes.c_longlong(0)
    ms = ctypes.c_double(0.0)
    _check(lib().ra_trace_query(k, ctypes.addressof(n), ctypes.addressof(ms)))
    return n.value, ms.value
