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
_CT = {"P": ctypes.c_void_p, "L": ctypes.c_longlong, "i": ctypes.c_int, "s": ctypes.c_char_p,
       "f": ctypes.c_float}


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
        out = torch.empty_like(o)
    if lse is None:
        lse = torch.empty_like(m)
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
        out = torch.empty((N, heads, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((N, heads), dtype=torch.float32, device=q.device)
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
        out = torch.empty((N, heads, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((N, heads), dtype=torch.float32, device=q.device)
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
        dq = torch.empty((N, heads, d), dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty((N, kv_heads, d), dtype=torch.float32, device=q.device)
    if dv is None:
        dv = torch.empty((N, kv_heads, d), dtype=torch.float32, device=q.device)
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
        dq = torch.empty((N, heads, d), dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty((N, kv_heads, d), dtype=torch.float32, device=q.device)
    if dv is None:
        dv = torch.empty((N, kv_heads, d), dtype=torch.float32, device=q.device)
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
        out = torch.empty((n_q, heads, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((n_q, heads), dtype=torch.float32, device=q.device)
    _state_shapes(lse, lse, out, n_q, heads, d)
    kp = _dev(k, "k") if n_kv else 0
    vp = _dev(v, "v") if n_kv else 0
    _check(lib().ra_decode_forward(
        _dev(q, "q"), kp, vp, _dev(out, "out", torch.float32), _dev(lse, "lse", torch.float32),
        n_q, n_kv, int(P), int(q_off), int(bool(causal)), int(window), d, heads, kv_heads,
        _qkv_dtype(q), _stream(stream)))
    return out, lse


# ------------------------------------------------------------------ rotary positions, pages

# These calls are made once or more per layer of a serving step, where a few
# microseconds of Python each are the step's time: their checks read every
# tensor property once, and the device is switched only when it must be.

def _device(t, name) -> int:
    """Index of the CUDA device a tensor lives on."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _arg(t, name, dev, dtype):
    """Pointer of a dense tensor of `dtype` on device `dev`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor" if t.get_device() < 0 else
                         f"{name} is on {t.device}, not on cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _vec(t, name, n, dev, dtype):
    """Pointer of a dense 1-D tensor of n entries."""
    p = _arg(t, name, dev, dtype)
    if t.dim() != 1 or t.numel() != n:
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    return p


def _rows(t, name, T, heads, d, dev, dtype):
    """Pointer and token stride of a [T, heads, d] tensor whose heads are
    dense; tokens may lie further apart (a view of a packed projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor" if t.get_device() < 0 else
                         f"{name} is on {t.device}, not on cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    st = t.stride()
    if T and (st[2] != 1 or (heads > 1 and st[1] != d)):
        raise ValueError(f"{name}: the heads of a token must be dense (strides {st})")
    return t.data_ptr(), st[0] if T > 1 else heads * d


def _call(name, dev, stream, *args):
    """Call a library function with device `dev` current, on `stream` (None:
    the device's current stream), the last argument."""
    f = getattr(_lib or lib(), name)
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == dev:
        rc = f(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, st)
    if rc:
        _check(rc)


def _weights(q_weight, k_weight, d, dev):
    """Pointers of the norm weights (0 for none) and their dtype."""
    code, ptrs = RA_F32, []
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is None:
            ptrs.append(0)
            continue
        if w.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{name} must be float32 or bfloat16, got {w.dtype}")
        ptrs.append(_vec(w, name, d, dev, w.dtype))
        if w.dtype is torch.bfloat16:
            code = RA_BF16
    if q_weight is not None and k_weight is not None and q_weight.dtype is not k_weight.dtype:
        raise TypeError("q_weight and k_weight must share a dtype")
    return ptrs[0], ptrs[1], code


def _phase_table(phases, dev):
    if phases is None:
        return 0, 0
    n = phases.numel()
    return _vec(phases, "phases", n, dev, torch.int64), 2 * n


def _qk_shapes(q, k):
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError("q: [T, heads, d]; k: [T, kv_heads, d]")
    if ks[0] != qs[0] or ks[2] != qs[2] or k.dtype is not q.dtype:
        raise ValueError("q and k must share their tokens, head dim and dtype")
    return qs[0], qs[1], ks[1], qs[2]


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
    T, heads, kv_heads, d = _qk_shapes(q, k)
    dt = _qkv_dtype(q)
    if q_out is None:
        q_out = torch.empty((T, heads, d), dtype=q.dtype, device=q.device)
    elif q_out.shape != q.shape:
        raise ValueError("q_out and k_out must match q and k in shape")
    if k_out is None:
        k_out = torch.empty((T, kv_heads, d), dtype=q.dtype, device=q.device)
    elif k_out.shape != k.shape:
        raise ValueError("q_out and k_out must match q and k in shape")
    dev, dtype = _device(q, "q"), q.dtype
    qp, qs = _rows(q, "q", T, heads, d, dev, dtype)
    kp, ks = _rows(k, "k", T, kv_heads, d, dev, dtype)
    ph, rot = _phase_table(phases, dev)
    qw, kw, wt = _weights(q_weight, k_weight, d, dev)
    pos = 0 if positions is None else _vec(positions, "positions", T, dev, torch.int32)
    _call("ra_qk_norm_rope", dev, stream,
        qp, kp, _arg(q_out, "q_out", dev, dtype), _arg(k_out, "k_out", dev, dtype), T, d,
        heads, kv_heads, qs, ks, pos, _layout(layout), int(P), rot, int(bool(interleaved)),
        ph, float(mscale), qw, kw, wt, float(eps), dt)
    return q_out, k_out


def ra_qk_norm_rope_backward(q, k, phases, dq_out, dk_out, *, q_weight=None, k_weight=None,
                             eps: float = 1e-6, interleaved: bool = False, mscale: float = 1.0,
                             positions=None, P: int = 1, layout="contiguous", dq=None, dk=None,
                             dq_weight=None, dk_weight=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ra_qk_norm_rope's inputs
    from those of its outputs (fp32, dense, as ra_ring_backward returns
    them).  dq and dk have q's dtype and may be views of a packed gradient;
    the weights' are fp32 [d], None without that weight."""
    T, heads, kv_heads, d = _qk_shapes(q, k)
    dt = _qkv_dtype(q)
    if dq_out.shape != q.shape or dk_out.shape != k.shape:
        raise ValueError("dq_out and dk_out must match q and k in shape")
    if dq is None:
        dq = torch.empty((T, heads, d), dtype=q.dtype, device=q.device)
    if dk is None:
        dk = torch.empty((T, kv_heads, d), dtype=q.dtype, device=q.device)
    if dq.shape != q.shape or dk.shape != k.shape:
        raise ValueError("dq and dk must match q and k in shape")
    for w, g, name in ((q_weight, dq_weight, "dq_weight"), (k_weight, dk_weight, "dk_weight")):
        if w is None and g is not None:
            raise ValueError(f"{name} without its weight")
    if q_weight is not None and dq_weight is None:
        dq_weight = torch.empty(d, dtype=torch.float32, device=q.device)
    if k_weight is not None and dk_weight is None:
        dk_weight = torch.empty(d, dtype=torch.float32, device=q.device)
    dev, dtype, f32 = _device(q, "q"), q.dtype, torch.float32
    qp, qs = _rows(q, "q", T, heads, d, dev, dtype)
    kp, ks = _rows(k, "k", T, kv_heads, d, dev, dtype)
    dqp, dqs = _rows(dq, "dq", T, heads, d, dev, dtype)
    dkp, dks = _rows(dk, "dk", T, kv_heads, d, dev, dtype)
    ph, rot = _phase_table(phases, dev)
    qw, kw, wt = _weights(q_weight, k_weight, d, dev)
    pos = 0 if positions is None else _vec(positions, "positions", T, dev, torch.int32)
    dqw = 0 if dq_weight is None else _vec(dq_weight, "dq_weight", d, dev, f32)
    dkw = 0 if dk_weight is None else _vec(dk_weight, "dk_weight", d, dev, f32)
    _call("ra_qk_norm_rope_backward", dev, stream,
        qp, kp, _arg(dq_out, "dq_out", dev, f32), _arg(dk_out, "dk_out", dev, f32), dqp, dkp,
        dqw, dkw, T, d, heads, kv_heads, qs, ks, dqs, dks, pos, _layout(layout), int(P), rot,
        int(bool(interleaved)), ph, float(mscale), qw, kw, wt, float(eps), dt)
    return dq, dk, dq_weight, dk_weight


def _table(block_table, n_req, dev):
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != n_req:
        raise ValueError(f"block_table must be [n_req={n_req}, max_pages], got {tuple(shape)}")
    return _arg(block_table, "block_table", dev, torch.int32), shape[1]


def ra_paged_extend(lengths, new_tokens, block_table, free_pages, free_count, *, page_size: int,
                    tokens: int, lengths_out=None, free_count_out=None, slots=None,
                    positions=None, cu_tokens=None, status=None, stream=None):
    """Hand out pages for a step's new tokens (all on the device, int32 but
    for slots): block_table's rows are extended in place, and the call
    returns (slots int64 [tokens], positions [tokens], cu_tokens [n_req + 1],
    lengths_out [n_req], free_count_out [1], status [3]).  lengths_out and
    free_count_out may be lengths and free_count themselves.  A nonzero
    status (pages missing, rows too short, tokens beyond `tokens`) means
    that the step changed nothing."""
    n, tokens = lengths.numel(), int(tokens)
    i32 = torch.int32
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError(f"block_table must be [n_req={n}, max_pages], "
                         f"got {tuple(block_table.shape)}")
    dev = _device(lengths, "lengths")
    where = lengths.device
    if lengths_out is None:
        lengths_out = torch.empty(n, dtype=i32, device=where)
    if free_count_out is None:
        free_count_out = torch.empty(1, dtype=i32, device=where)
    if slots is None:
        slots = torch.empty(tokens, dtype=torch.int64, device=where)
    if positions is None:
        positions = torch.empty(tokens, dtype=i32, device=where)
    if cu_tokens is None:
        cu_tokens = torch.empty(n + 1, dtype=i32, device=where)
    if status is None:
        status = torch.empty(3, dtype=i32, device=where)
    table, width = _table(block_table, n, dev)
    pool = free_pages.numel()
    _call("ra_paged_extend", dev, stream,
        _vec(lengths, "lengths", n, dev, i32), _vec(new_tokens, "new_tokens", n, dev, i32), n,
        table, width, _vec(free_pages, "free_pages", pool, dev, i32), pool,
        _vec(free_count, "free_count", 1, dev, i32), int(page_size), tokens,
        _vec(lengths_out, "lengths_out", n, dev, i32),
        _vec(free_count_out, "free_count_out", 1, dev, i32),
        _vec(slots, "slots", tokens, dev, torch.int64),
        _vec(positions, "positions", tokens, dev, i32),
        _vec(cu_tokens, "cu_tokens", n + 1, dev, i32), _vec(status, "status", 3, dev, i32))
    return slots, positions, cu_tokens, lengths_out, free_count_out, status


def ra_paged_release(lengths, finished, block_table, free_pages, free_count, *, page_size: int,
                     lengths_out=None, free_count_out=None, stream=None):
    """Push the pages of the requests with finished != 0 back on the stack
    free_pages (in place) and set their lengths to 0; returns (lengths_out,
    free_count_out), which may be lengths and free_count themselves."""
    n, i32 = lengths.numel(), torch.int32
    dev = _device(lengths, "lengths")
    if lengths_out is None:
        lengths_out = torch.empty(n, dtype=i32, device=lengths.device)
    if free_count_out is None:
        free_count_out = torch.empty(1, dtype=i32, device=lengths.device)
    table, width = _table(block_table, n, dev)
    pool = free_pages.numel()
    _call("ra_paged_release", dev, stream,
        _vec(lengths, "lengths", n, dev, i32), _vec(finished, "finished", n, dev, i32), n,
        table, width, _vec(free_pages, "free_pages", pool, dev, i32), pool,
        _vec(free_count, "free_count", 1, dev, i32), int(page_size),
        _vec(lengths_out, "lengths_out", n, dev, i32),
        _vec(free_count_out, "free_count_out", 1, dev, i32))
    return lengths_out, free_count_out


def _cache(t, name, kv_heads, d, dev):
    """Pointer, page count, page size and page stride of a cache tensor
    [n_pages, page_size, kv_heads, d] (bf16, dense inside a page)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor" if t.get_device() < 0 else
                         f"{name} is on {t.device}, not on cuda:{dev}")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 4 or shape[2] != kv_heads or shape[3] != d:
        raise ValueError(f"{name} must be [n_pages, page_size, {kv_heads}, {d}], "
                         f"got {tuple(shape)}")
    n, ps = shape[0], shape[1]
    st = t.stride()
    if n and (st[3] != 1 or (kv_heads > 1 and st[2] != d) or (ps > 1 and st[1] != kv_heads * d)):
        raise ValueError(f"{name}: a page must be dense (strides {st})")
    return t.data_ptr(), n, ps, st[0] if n > 1 else ps * kv_heads * d


def _caches(k_cache, v_cache, kv_heads, d, dev):
    kp, n, ps, ks = _cache(k_cache, "k_cache", kv_heads, d, dev)
    vp, vn, vps, vs = _cache(v_cache, "v_cache", kv_heads, d, dev)
    if vn != n or vps != ps:
        raise ValueError("k_cache and v_cache must match in pages and page size")
    return kp, vp, n, ps, ks, vs


def ra_paged_append(q, k, v, phases, k_cache, v_cache, slots, positions, *, q_weight=None,
                    k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                    mscale: float = 1.0, q_out=None, stream=None):
    """ra_qk_norm_rope on a step's rows (bf16) with k and v written to their
    pages: row t goes to slots[t] (int64; outside the pages: padding, nothing
    is written) at positions[t] (int32).  Returns q_out, dense like q."""
    T, heads, kv_heads, d = _qk_shapes(q, k)
    dt = _qkv_dtype(q)
    if v.shape != k.shape or v.dtype is not q.dtype:
        raise ValueError("v must match k in shape and dtype")
    if q_out is None:
        q_out = torch.empty((T, heads, d), dtype=q.dtype, device=q.device)
    elif q_out.shape != q.shape:
        raise ValueError("q_out must match q in shape")
    dev, dtype = _device(q, "q"), q.dtype
    qp, qs = _rows(q, "q", T, heads, d, dev, dtype)
    kp, ks = _rows(k, "k", T, kv_heads, d, dev, dtype)
    vp, vs = _rows(v, "v", T, kv_heads, d, dev, dtype)
    kc, vc, n_pages, ps, kcs, vcs = _caches(k_cache, v_cache, kv_heads, d, dev)
    ph, rot = _phase_table(phases, dev)
    qw, kw, wt = _weights(q_weight, k_weight, d, dev)
    _call("ra_paged_append", dev, stream,
        qp, kp, vp, _arg(q_out, "q_out", dev, dtype), kc, vc, T, d, heads, kv_heads, qs, ks,
        vs, n_pages, ps, kcs, vcs, _vec(slots, "slots", T, dev, torch.int64),
        _vec(positions, "positions", T, dev, torch.int32), rot, int(bool(interleaved)), ph,
        float(mscale), qw, kw, wt, float(eps), dt)
    return q_out


def ra_paged_decode(q, k_cache, v_cache, block_table, lengths, *, cu_q=None, window: int = 0,
                    out=None, lse=None, stream=None):
    """Attention of each request's newest tokens q [T, heads, d] (bf16) over
    its pages.  T / n_req rows per request, or rows [cu_q[i], cu_q[i + 1]) of
    request i (int32 [n_req + 1]); lengths (int32 [n_req]) include them.
    Returns (out [T, heads, d], lse [T, heads]), fp32; pass a bf16 `out` for
    that type."""
    n = lengths.numel()
    if q.dim() != 3:
        raise ValueError("q: [T, heads, d]")
    T, heads, d = q.shape
    if k_cache.dim() != 4:
        raise ValueError("k_cache: [n_pages, page_size, kv_heads, d]")
    kv_heads = k_cache.shape[2]
    if cu_q is None and (T % n if n else T):
        raise ValueError(f"T={T} rows are not a multiple of {n} requests (and cu_q is None)")
    f32 = torch.float32
    if out is None:
        out = torch.empty((T, heads, d), dtype=f32, device=q.device)
    elif out.shape != q.shape:
        raise ValueError(f"out must have shape {(T, heads, d)}, got {tuple(out.shape)}")
    elif out.dtype not in (f32, torch.bfloat16):
        raise TypeError(f"out must be float32 or bfloat16, got {out.dtype}")
    if lse is None:
        lse = torch.empty((T, heads), dtype=f32, device=q.device)
    elif tuple(lse.shape) != (T, heads):
        raise ValueError(f"lse must have shape {(T, heads)}, got {tuple(lse.shape)}")
    dev = _device(q, "q")
    kc, vc, n_pages, ps, ks, vs = _caches(k_cache, v_cache, kv_heads, d, dev)
    table, width = _table(block_table, n, dev)
    cu = 0 if cu_q is None else _vec(cu_q, "cu_q", n + 1, dev, torch.int32)
    _call("ra_paged_decode", dev, stream,
        _arg(q, "q", dev, torch.bfloat16), kc, vc, _arg(out, "out", dev, out.dtype),
        _arg(lse, "lse", dev, f32), T, n, 0 if cu or not n else T // n, cu, table, width,
        _vec(lengths, "lengths", n, dev, torch.int32), n_pages, ps, ks, vs, int(window), d,
        heads, kv_heads, RA_BF16, RA_BF16 if out.dtype is torch.bfloat16 else RA_F32)
    return out, lse


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
        out = torch.empty((N, heads, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((N, heads), dtype=torch.float32, device=q.device)
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
