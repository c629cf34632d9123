"""ctypes binding of libfa_gb300.so (include/fa.h).

Argument marshalling only: torch tensors are checked for dtype, device and
layout, and their data pointers are handed to the C entry points, which run
every step on the GPU.  There is no fallback: if the library is missing or a
call fails, a ``FaError`` is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa_gb300.so")

FA_F16, FA_BF16 = 0, 1
(FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_WORKSPACE,
 FA_ERR_CACHE) = range(7)

# Symbols include/fa.h declares, with their ctypes signatures.
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fa_fwd_qk": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fa_fwd_splitkv": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _i, _vp,
                            _sz, _vp]),
    "fa_fwd_splitkv_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "fa_bwd_qk": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f,
                       _i, _i, _vp, _sz, _vp]),
    "fa_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_bwd_workspace_size_for": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i,
                    _vp, _sz, _vp]),
    "fa_bwd_deterministic": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                  _i, _f, _i, _vp, _sz, _vp]),
    "fa_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f,
                            _i, _vp]),
    "fa_fwd_blocksparse": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp,
                                _i, _vp]),
    "fa_bwd_blocksparse": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                _i, _f, _i, _vp, _i, _i, _vp, _sz, _vp]),
    "fa_fwd_strided": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "fa_bwd_strided": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                            _f, _i, _vp, _i, _vp, _sz, _vp]),
    "fa_rope": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _i, _i, _vp, _vp]),
    "fa_cache_append": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp,
                             _vp]),
    "fa_fwd_cache": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp, _vp, _sz,
                          _vp]),
    "fa_fwd_cache_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_get_device_status": (_i, [_vp]),
    "fa_strerror": (ctypes.c_char_p, [_i]),
    "fa_selftest_expired_wait": (_i, [_i, _vp]),
    "fa_measure_ex2_rate": (_i, [ctypes.POINTER(ctypes.c_double), _vp]),
    "fa_measure_reduce_rate": (_i, [_vp, _sz, ctypes.POINTER(ctypes.c_double), _vp]),
    "fa_timing_enable": (_i, [_i]),
    "fa_timing_read": (_i, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)]),
}
KERNEL_KINDS = ("fwd", "bwd_pre", "bwd_main", "bwd_convert", "bwd_dq")

_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what} failed with status {status}: {strerror(status)}")


def load(path: str = LIB_PATH):
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise FaError(-1, f"loading {path}: library not built (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def strerror(status: int) -> str:
    try:
        return load().fa_strerror(status).decode()
    except Exception:
        return "library not loaded"


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return FA_F16
    if t.dtype == torch.bfloat16:
        return FA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; fp16 and bf16 are supported")


def _stream_ptr(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream or None


def _check(st: int, what: str):
    if st != FA_OK:
        raise FaError(st, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------- raw entry points
def fa_fwd(q, k, v, o, lse, B, H, Hkv, N, d, causal, scale, dtype, stream=None) -> int:
    return load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, N, d,
                         int(causal), float(scale), dtype, _stream_ptr(stream))


def fa_bwd_workspace_size(B, H, Hkv, N, d) -> int:
    return int(load().fa_bwd_workspace_size(B, H, Hkv, N, d))


def fa_bwd_workspace_size_for(B, H, Hkv, Nq, d, deterministic) -> int:
    return int(load().fa_bwd_workspace_size_for(B, H, Hkv, Nq, d, int(bool(deterministic))))


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, N, d, causal, scale, dtype, workspace,
           workspace_bytes, stream=None) -> int:
    return load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                         _ptr(dk), _ptr(dv), B, H, Hkv, N, d, int(causal), float(scale), dtype,
                         _ptr(workspace), int(workspace_bytes), _stream_ptr(stream))


def fa_bwd_deterministic(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, N, d, causal, scale, dtype,
                         workspace, workspace_bytes, stream=None) -> int:
    return load().fa_bwd_deterministic(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                       _ptr(dq), _ptr(dk), _ptr(dv), B, H, Hkv, N, d, int(causal),
                                       float(scale), dtype, _ptr(workspace), int(workspace_bytes),
                                       _stream_ptr(stream))


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, N, d, causal, scale, dtype,
                   stream=None) -> int:
    """fa_bwd with the library's own fixed device scratch (no allocation)."""
    return load().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, H, Hkv, N, d, int(causal),
                                 float(scale), dtype, _stream_ptr(stream))


def fa_get_device_status(stream=None) -> int:
    return load().fa_get_device_status(_stream_ptr(stream))


# ---------------------------------------------------------------- tensor helpers
class FaStrides(ctypes.Structure):
    """struct fa_strides: element strides (batch, head, row) of a [B][heads][N][d] view."""
    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong),
                ("row", ctypes.c_longlong)]


def _shapes(q, k, v, contiguous=True):
    """(B, H, Hkv, Nq, Nk, d) of q [B,H,Nq,d], k and v [B,Hkv,Nk,d] (views with
    the last dimension contiguous are accepted when contiguous=False)."""
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("expected q [B,H,Nq,d], k and v [B,Hkv,Nk,d]")
    B, H, Nq, d = q.shape
    if k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)}")
    for t in (q, k, v):
        if not t.is_cuda or t.dtype != q.dtype:
            raise ValueError("q, k, v must be CUDA tensors of one dtype")
        if contiguous and not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
        if not contiguous and t.stride(3) != 1:
            raise ValueError("the last (d) dimension must be contiguous")
    return B, H, k.shape[1], Nq, k.shape[2], d


def _strides(*ts):
    """fa_strides[len(ts)] of [B, heads, N, d] views (d contiguous)."""
    arr = (FaStrides * len(ts))()
    for i, t in enumerate(ts):
        if t.dim() != 4 or t.stride(3) != 1:
            raise ValueError("expected a [B, heads, N, d] view with d contiguous")
        arr[i] = FaStrides(t.stride(0), t.stride(1), t.stride(2))
    return arr


def forward_strided(q, k, v, causal: bool, scale: float, out=None, lse=None, stream=None):
    """fa_fwd_strided: q [B,H,Nq,d], k, v [B,Hkv,Nk,d] given as any views whose
    d elements are contiguous (e.g. x.transpose(1, 2) of a [B, N, H, d]
    tensor); out (allocated like q's layout unless given) likewise.  Returns
    (o, lse)."""
    B, H, Hkv, Nq, Nk, d = _shapes(q, k, v, contiguous=False)
    if out is None:
        out = torch.empty_like(q)   # same strides as q when q is dense in memory
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    _check(load().fa_fwd_strided(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, Nq,
                                 Nk, d, int(causal), float(scale), _dtype_code(q),
                                 _strides(q, k, v, out), _stream_ptr(stream)), "fa_fwd_strided")
    return out, lse


def backward_strided(q, k, v, o, lse, dout, causal: bool, scale: float, dq=None, dk=None,
                     dv=None, workspace=None, stream=None, deterministic: bool = False):
    """fa_bwd_strided: the gradients of forward_strided; every tensor may be a
    strided view (d contiguous); dq, dk, dv are allocated like q, k, v unless
    given.  Returns (dq, dk, dv)."""
    B, H, Hkv, Nq, Nk, d = _shapes(q, k, v, contiguous=False)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = fa_bwd_workspace_size_for(B, H, Hkv, Nq, d, deterministic)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check(load().fa_bwd_strided(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, H, Hkv, Nq, Nk, d, int(causal),
                                 float(scale), _dtype_code(q),
                                 _strides(q, k, v, o, dout, dq, dk, dv), int(bool(deterministic)),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream)), "fa_bwd_strided")
    return dq, dk, dv


def forward(q, k, v, causal: bool, scale: float, out=None, lse=None, stream=None):
    """(o, lse) of exact attention; outputs are allocated unless given.  The
    key length may differ from the query length (causal mask bottom-right)."""
    B, H, Hkv, Nq, Nk, d = _shapes(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if Nq == Nk:
        st = fa_fwd(q, k, v, out, lse, B, H, Hkv, Nq, d, causal, scale, _dtype_code(q), stream)
    else:
        st = load().fa_fwd_qk(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, Nq, Nk,
                              d, int(causal), float(scale), _dtype_code(q), _stream_ptr(stream))
    _check(st, "fa_fwd")
    return out, lse


def backward(q, k, v, o, lse, dout, causal: bool, scale: float, dq=None, dk=None, dv=None,
             workspace=None, stream=None, deterministic: bool = False):
    """(dq, dk, dv) of sum(O o dO); outputs and scratch are allocated unless given.
    deterministic=True uses fa_bwd_deterministic (bitwise reproducible dQ)."""
    B, H, Hkv, Nq, Nk, d = _shapes(q, k, v)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = fa_bwd_workspace_size_for(B, H, Hkv, Nq, d, deterministic)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if Nq == Nk:
        fn = fa_bwd_deterministic if deterministic else fa_bwd
        st = fn(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, Nq, d, causal, scale,
                _dtype_code(q), workspace, ws_bytes, stream)
    else:
        st = load().fa_bwd_qk(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, H, Hkv, Nq, Nk, d, int(causal), float(scale),
                              _dtype_code(q), int(bool(deterministic)), _ptr(workspace),
                              ws_bytes, _stream_ptr(stream))
    _check(st, "fa_bwd_deterministic" if deterministic else "fa_bwd")
    return dq, dk, dv


def device_status(stream=None):
    """Synchronise the stream and raise if a kernel reported a bounded-wait timeout."""
    _check(fa_get_device_status(stream), "fa_get_device_status")


def measure_ex2_rate(stream=None) -> float:
    """Exponentials per second of the device's ex2 unit (fa_measure_ex2_rate)."""
    out = ctypes.c_double(0.0)
    _check(load().fa_measure_ex2_rate(ctypes.byref(out), _stream_ptr(stream)),
           "fa_measure_ex2_rate")
    return out.value


def measure_reduce_rate(scratch: torch.Tensor, stream=None) -> float:
    """Bytes per second of fp32 bulk reduce-adds from every SM into `scratch`
    (a device tensor of at least 1 MiB, 256-byte aligned; zeros are added:
    fa_measure_reduce_rate)."""
    out = ctypes.c_double(0.0)
    _check(load().fa_measure_reduce_rate(ctypes.c_void_p(scratch.data_ptr()),
                                         scratch.numel() * scratch.element_size(),
                                         ctypes.byref(out), _stream_ptr(stream)),
           "fa_measure_reduce_rate")
    return out.value


def timing_enable(capacity: int):
    """Start (capacity > 0) or stop (0) per-kernel event timing inside the library."""
    _check(load().fa_timing_enable(int(capacity)), "fa_timing_enable")


def timing_read():
    """{kind: (summed ms, launches)} of the kernels timed since the last read."""
    ms = (ctypes.c_double * len(KERNEL_KINDS))()
    n = (ctypes.c_int * len(KERNEL_KINDS))()
    _check(load().fa_timing_read(ms, n), "fa_timing_read")
    return {k: (ms[i], n[i]) for i, k in enumerate(KERNEL_KINDS)}


def forward_splitkv(q, k, v, causal: bool, scale: float, num_splits: int = 0, out=None, lse=None,
                    workspace=None, stream=None):
    """(o, lse) through fa_fwd_splitkv (key axis split, partials merged on the GPU)."""
    B, H, Hkv, Nq, Nk, d = _shapes(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    need = int(load().fa_fwd_splitkv_workspace_size(B, H, Hkv, Nq, Nk, d, int(num_splits)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(load().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, Nq,
                                 Nk, d, int(causal), float(scale), _dtype_code(q), int(num_splits),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream)), "fa_fwd_splitkv")
    return out, lse


def _check_mask(block_mask, H, Nq, Nk, device):
    """A block mask [1 or H, ceil(Nq/128), ceil(Nk/128)] as a contiguous uint8
    CUDA tensor (nonzero = computed); returns (mask, mask_heads)."""
    nbr, nbc = -(-Nq // 128), -(-Nk // 128)
    if (block_mask.dim() != 3 or block_mask.shape[0] not in (1, H)
            or tuple(block_mask.shape[1:]) != (nbr, nbc)):
        raise ValueError(f"block mask must be [1 or {H}, {nbr}, {nbc}], got "
                         f"{tuple(block_mask.shape)}")
    if block_mask.dtype not in (torch.uint8, torch.bool):
        raise TypeError("block mask must be uint8 or bool")
    if not block_mask.is_cuda or block_mask.device != device or not block_mask.is_contiguous():
        raise ValueError("block mask must be a contiguous tensor on the inputs' device")
    return block_mask, int(block_mask.shape[0])


def forward_blocksparse(q, k, v, block_mask, causal: bool, scale: float, out=None, lse=None,
                        stream=None):
    """(o, lse) of exact attention restricted to the kept 128 x 128 blocks of
    block_mask [1 or H, ceil(Nq/128), ceil(Nk/128)] (fa_fwd_blocksparse)."""
    B, H, Hkv, Nq, Nk, d = _shapes(q, k, v)
    mask, mh = _check_mask(block_mask, H, Nq, Nk, q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    _check(load().fa_fwd_blocksparse(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv,
                                     Nq, Nk, d, int(causal), float(scale), _dtype_code(q),
                                     _ptr(mask), mh, _stream_ptr(stream)), "fa_fwd_blocksparse")
    return out, lse


def backward_blocksparse(q, k, v, o, lse, dout, block_mask, causal: bool, scale: float, dq=None,
                         dk=None, dv=None, workspace=None, stream=None,
                         deterministic: bool = False):
    """(dq, dk, dv) of the block-sparse forward above (fa_bwd_blocksparse)."""
    B, H, Hkv, Nq, Nk, d = _shapes(q, k, v)
    mask, mh = _check_mask(block_mask, H, Nq, Nk, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = fa_bwd_workspace_size_for(B, H, Hkv, Nq, d, deterministic)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check(load().fa_bwd_blocksparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                     _ptr(dq), _ptr(dk), _ptr(dv), B, H, Hkv, Nq, Nk, d,
                                     int(causal), float(scale), _dtype_code(q), _ptr(mask), mh,
                                     int(bool(deterministic)), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _stream_ptr(stream)), "fa_bwd_blocksparse")
    return dq, dk, dv


# ---------------------------------------------------------------- rotary positions, 8-bit cache
ROPE_MAX_PAIRS, ROPE_MAX_AXES = 128, 4


class _FaRopeSpec(ctypes.Structure):
    """struct fa_rope_spec"""
    _fields_ = [("axes", ctypes.c_int), ("pairs", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("freq", ctypes.c_double * ROPE_MAX_PAIRS),
                ("axis", ctypes.c_ubyte * ROPE_MAX_PAIRS)]


class _FaCache(ctypes.Structure):
    """struct fa_cache"""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("block_table", _vp),
                ("pages", _i), ("page_size", _i), ("table_width", _i), ("Hkv", _i), ("d", _i),
                ("k_strides", FaStrides), ("v_strides", FaStrides)]


class Rope:
    """The angles of a rotation (struct fa_rope_spec): pair p turns by freq[p]
    radians per position of axis axis[p] (all on one axis unless given).
    freq: a sequence of numbers or a tensor, read once, here."""

    def __init__(self, freq, axis=None, interleaved: bool = False):
        freq = [float(f) for f in freq]
        axis = [0] * len(freq) if axis is None else [int(a) for a in axis]
        if not 1 <= len(freq) <= ROPE_MAX_PAIRS or len(axis) != len(freq):
            raise ValueError(f"expected 1 to {ROPE_MAX_PAIRS} frequencies and an axis for each")
        if min(axis) < 0 or max(axis) >= ROPE_MAX_AXES:
            raise ValueError(f"axes are numbered 0 to {ROPE_MAX_AXES - 1}")
        self.axes, self.pairs = max(axis) + 1, len(freq)
        self.spec = _FaRopeSpec(axes=self.axes, pairs=self.pairs, interleaved=int(bool(interleaved)))
        self.spec.freq[:self.pairs] = freq
        self.spec.axis[:self.pairs] = axis
        self._ref = ctypes.addressof(self.spec)


class Cache:
    """A paged 8-bit key/value cache (struct fa_cache): k, v
    [pages, Hkv, page_size, d] of torch.float8_e4m3fn (or their bytes as
    uint8; any view with d contiguous), k_scale, v_scale fp32 [pages, Hkv],
    block_table int32 [B, table_width].  The tensors are the caller's; the
    object keeps them alive and holds their addresses."""

    def __init__(self, k, v, k_scale, v_scale, block_table):
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("expected k and v [pages, Hkv, page_size, d]")
        pages, Hkv, page, d = k.shape
        for t in (k, v):
            if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise TypeError("the cache's k and v are float8_e4m3fn (or uint8 codes)")
            if t.stride(3) != 1:
                raise ValueError("the last (d) dimension must be contiguous")
        for t in (k_scale, v_scale):
            if t.dtype != torch.float32 or tuple(t.shape) != (pages, Hkv) or not t.is_contiguous():
                raise ValueError(f"scales must be contiguous fp32 [{pages}, {Hkv}]")
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
            raise ValueError("block_table must be contiguous int32 [B, table_width]")
        self.tensors = (k, v, k_scale, v_scale, block_table)
        if any(not t.is_cuda or t.device != k.device for t in self.tensors):
            raise ValueError("the cache's tensors must be on one CUDA device")
        self.pages, self.Hkv, self.page_size, self.d = pages, Hkv, page, d
        self.B, self.table_width = block_table.shape
        self.device, self.device_index = k.device, k.get_device()
        self.key = (self.B, Hkv, d, self.device_index)
        self.struct = _FaCache(*(t.data_ptr() for t in self.tensors), pages, page, self.table_width,
                               Hkv, d, _view_strides(k), _view_strides(v))
        self._ref = ctypes.addressof(self.struct)


def _view_strides(t):
    """FaStrides of a [.., .., .., d] view; a dimension of one element has no
    stride of its own and takes the contiguous one."""
    s = t.stride()
    n = t.shape
    row = s[2] if n[2] > 1 else n[3]
    head = s[1] if n[1] > 1 else n[2] * n[3]
    batch = s[0] if n[0] > 1 else n[1] * n[2] * n[3]
    return FaStrides(batch, head, row)


_L6, _L12 = ctypes.c_longlong * 6, ctypes.c_longlong * 12   # two and four fa_strides
_plans: dict = {}   # what a call's shapes, strides, types and device come to, checked once


def _plan(make, *key):
    """make(*key), kept: a call's checks and stride arrays depend on its
    tensors' geometry alone, and a decoding loop repeats the same few."""
    key = (make, *key)
    plan = _plans.get(key)
    if plan is None:
        plan = make(*key[1:])
        if len(_plans) >= 512:
            _plans.clear()
        _plans[key] = plan
    return plan


def _geometry(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _view(geometry, shape, dtype, device, what):
    """(batch, head, row) strides of a [B, heads, N, d] view that has to be of
    the shape, dtype and device (an index) given."""
    of, s, its_dtype, its_device = geometry
    if of != shape:
        raise ValueError(f"{what}: shape {tuple(of)}, expected {tuple(shape)}")
    if its_dtype != dtype or its_device != device:
        raise ValueError(f"{what} must have the dtype and device of the other tensors")
    B, heads, N, d = shape
    if s[3] != 1:
        raise ValueError("the last (d) dimension must be contiguous")
    # a dimension of one element has no stride of its own
    return (s[0] if B > 1 else heads * N * d, s[1] if heads > 1 else N * d, s[2] if N > 1 else d)


def _code(dtype):
    if dtype == torch.float16:
        return FA_F16
    if dtype == torch.bfloat16:
        return FA_BF16
    raise TypeError(f"unsupported dtype {dtype}; fp16 and bf16 are supported")


def _ints(t, shape, device, what):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous int32 {list(shape)} on the inputs' device")
    return t.data_ptr()


def _positions(positions, axes, B, N, device):
    """(address, pos_batch) of positions [axes, B or 1, N] ([B or 1, N] on one axis)."""
    if positions is None:
        return None, 1
    shape = tuple(positions.shape)
    if len(shape) == 2 and axes == 1:
        shape = (1,) + shape
    if (positions.dtype != torch.int32 or len(shape) != 3 or shape[0] != axes or shape[1] not in (1, B)
            or shape[2] != N or positions.get_device() != device or not positions.is_contiguous()):
        raise ValueError(f"positions must be contiguous int32 [{axes}, {B} or 1, {N}] on the "
                         "inputs' device")
    return positions.data_ptr(), shape[1]


def _on_stream(device, stream, call, *args):
    """call(*args, raw stream) on the stream given, or on the current stream of
    the tensors' device (an index), which is made current for the call.  On a
    given stream everything the call allocates comes from that stream's memory,
    and its inputs are marked as used there, so that neither is handed out
    again before the call's work is done; what it returns is marked as used on
    the caller's stream too."""
    if device < 0:
        raise ValueError("expected CUDA tensors")
    if stream is None:
        if device == torch.cuda.current_device():
            return call(*args, torch._C._cuda_getCurrentRawStream(device) or None)
        with torch.cuda.device(device):
            return call(*args, torch._C._cuda_getCurrentRawStream(device) or None)
    if stream.device.index != device:
        raise ValueError("the stream belongs to another device than the tensors")
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = call(*args, stream.cuda_stream or None)
    if stream != caller:
        for a in args:
            for t in a.tensors if isinstance(a, Cache) else (a,):
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None:
                t.record_stream(caller)
    return out


def _rope_plan(q, k, q_out, k_out):
    if len(q[0]) != 4 or (k is not None and len(k[0]) != 4):
        raise ValueError("expected q [B, H, N, d] and k [B, Hkv, N, d]")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out belong together")
    B, H, N, d = q[0]
    Hkv = 0 if k is None else k[0][1]

    def view(t, heads, what):
        return (0, 0, 0) if t is None else _view(t, (B, heads, N, d), q[2], q[3], what)

    return B, H, Hkv, N, d, _code(q[2]), _L12(*view(q, H, "q"), *view(k, Hkv, "k"),
                                              *view(q_out, H, "q_out"), *view(k_out, Hkv, "k_out"))


def _rope(q, k, positions, table, inverse, q_out, k_out, stream):
    if q_out is None:
        q_out = torch.empty_like(q)
    if k is not None and k_out is None:
        k_out = torch.empty_like(k)
    B, H, Hkv, N, d, code, st = _plan(_rope_plan, _geometry(q), _geometry(k), _geometry(q_out),
                                      _geometry(k_out))
    pos, pos_batch = _positions(positions, table.axes, B, N, q.get_device())
    _check(load().fa_rope(q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out), B, H, Hkv, N, d, code,
                          table._ref, pos, pos_batch, inverse, st, stream), "fa_rope")
    return q_out, k_out


def rope(q, k, positions, table: Rope, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): q [B, H, N, d] and k [B, Hkv, N, d] (or None) rotated by
    `table` (fa_rope).  positions int32 [axes, B or 1, N] ([B or 1, N] on one
    axis), None: 0 .. N - 1.  Any views with d contiguous; outputs are
    allocated like the inputs unless given, and may be the inputs."""
    return _on_stream(q.get_device(), stream, _rope_forward, q, k, positions, table, q_out, k_out)


def rope_backward(dq_out, dk_out, positions, table: Rope, dq=None, dk=None, stream=None):
    """(dq, dk) of `rope` from the gradients of its outputs."""
    return _on_stream(dq_out.get_device(), stream, _rope_inverse, dq_out, dk_out, positions, table, dq,
                      dk)


def _rope_forward(q, k, positions, table, q_out, k_out, stream):
    return _rope(q, k, positions, table, 0, q_out, k_out, stream)


def _rope_inverse(q, k, positions, table, q_out, k_out, stream):
    return _rope(q, k, positions, table, 1, q_out, k_out, stream)


def cache_append(cache: Cache, q, k, v, seq_lens, new_lens=None, rope: Rope | None = None,
                 positions=None, q_out=None, stream=None):
    """Append the tokens k, v [B, Hkv, N, d] to the cache, keys rotated by
    `rope`, and return q [B, H, N, d] rotated (None for q None)
    (fa_cache_append).  seq_lens int32 [B]: lengths counting the new tokens;
    new_lens int32 [B]: how many of the N rows are tokens (None: all);
    positions as in `rope`, None: the tokens' numbers."""
    return _on_stream(k.get_device(), stream, _cache_append, cache, q, k, v, seq_lens, new_lens, rope,
                      positions, q_out)


def _append_plan(cache, q, k, v, q_out):
    if len(k[0]) != 4 or (q is not None and len(q[0]) != 4):
        raise ValueError("expected k and v [B, Hkv, N, d], q [B, H, N, d]")
    B, Hkv, N, d = k[0]
    if (B, Hkv, d, k[3]) != cache:
        raise ValueError(f"k{tuple(k[0])} does not belong to a cache of {cache[0]} sequences, "
                         f"{cache[1]} heads, d {cache[2]} on device {cache[3]}")
    H = 0 if q is None else q[0][1]

    def view(t, heads, what):
        return (0, 0, 0) if t is None else _view(t, (B, heads, N, d), k[2], k[3], what)

    return B, H, N, _code(k[2]), _L12(*view(q, H, "q"), *view(k, Hkv, "k"), *view(v, Hkv, "v"),
                                      *view(q_out, H, "q_out"))


def _cache_append(cache, q, k, v, seq_lens, new_lens, rope, positions, q_out, stream):
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = torch.empty_like(q)
    B, H, N, code, st = _plan(_append_plan, cache.key, _geometry(q), _geometry(k), _geometry(v),
                              _geometry(q_out))
    device = cache.device_index
    pos, pos_batch = _positions(positions, 1 if rope is None else rope.axes, B, N, device)
    _check(load().fa_cache_append(
        cache._ref, _ptr(q), k.data_ptr(), v.data_ptr(), _ptr(q_out), B, H, N, code,
        _ints(seq_lens, (B,), device, "seq_lens"), _ints(new_lens, (B,), device, "new_lens"),
        None if rope is None else rope._ref, pos, pos_batch, st, stream), "fa_cache_append")
    return q_out


def forward_cache(q, cache: Cache, seq_lens, causal: bool, scale: float, new_lens=None, out=None,
                  lse=None, workspace=None, stream=None):
    """(o, lse) of q [B, H, Nq, d] against the first seq_lens[b] tokens of the
    cache (fa_fwd_cache).  causal: the new_lens[b] query rows (None: all Nq)
    are the sequence's last tokens."""
    return _on_stream(q.get_device(), stream, _forward_cache, q, cache, seq_lens, causal, scale,
                      new_lens, out, lse, workspace)


def _forward_plan(cache, q, out):
    if len(q[0]) != 4:
        raise ValueError("expected q [B, H, Nq, d]")
    B, H, Nq, d = q[0]
    if (B, d, q[3]) != (cache[0], cache[2], cache[3]) or H % cache[1]:
        raise ValueError(f"q{tuple(q[0])} does not fit a cache of {cache[0]} sequences, {cache[1]} heads, "
                         f"d {cache[2]} on device {cache[3]}")
    return (B, H, Nq, _code(q[2]), _L6(*_view(q, q[0], q[2], q[3], "q"), *_view(out, q[0], q[2], q[3], "out")),
            fwd_cache_workspace_size(B, H, cache[1], Nq, d))


def _forward_cache(q, cache, seq_lens, causal, scale, new_lens, out, lse, workspace, stream):
    if out is None:
        out = torch.empty_like(q)
    B, H, Nq, code, st, ws_bytes = _plan(_forward_plan, cache.key, _geometry(q), _geometry(out))
    device = cache.device_index
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=cache.device)
    elif (lse.dtype != torch.float32 or lse.shape != (B, H, Nq) or lse.get_device() != device
          or not lse.is_contiguous()):
        raise ValueError(f"lse must be contiguous fp32 [{B}, {H}, {Nq}] on the inputs' device")
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=cache.device)
    else:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous and on the inputs' device")
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().fa_fwd_cache(
        q.data_ptr(), cache._ref, out.data_ptr(), lse.data_ptr(), B, H, Nq, int(causal), float(scale), code,
        _ints(seq_lens, (B,), device, "seq_lens"), _ints(new_lens, (B,), device, "new_lens"), st,
        workspace.data_ptr(), ws_bytes, stream), "fa_fwd_cache")
    return out, lse


def fwd_cache_workspace_size(B, H, Hkv, Nq, d) -> int:
    """Bytes of workspace forward_cache needs on the current device."""
    return int(load().fa_fwd_cache_workspace_size(B, H, Hkv, Nq, d))
