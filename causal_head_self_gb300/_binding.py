"""ctypes binding of libattn_sm103a.so (include/attn.h), same names as the
C ABI.  Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  torch is used for device memory and streams.

If the library has not been built the first call raises: there is no other
implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
import typing

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# CHS_ATTN_CHECK=1 selects the range-checked build of the same library
# (build.build(check=True)); it runs the same kernels with every copy they
# issue checked, a failed check reported as ATTN_ERR_CHECK
LIB_PATH = os.path.join(_PKG, "libattn_sm103a_check.so" if os.environ.get("CHS_ATTN_CHECK") == "1"
                        else "libattn_sm103a.so")

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_TIMEOUT = 4
ATTN_ERR_NO_MEMORY = 5
ATTN_ERR_SCRATCH_LIMIT = 6
ATTN_ERR_CHECK = 7

# every symbol include/attn.h declares
ABI_SYMBOLS = ("attn_fwd", "attn_fwd_lse", "attn_fwd_chunk", "attn_bwd", "attn_decode",
               "attn_decode_ring", "attn_decode_noalloc", "attn_status", "attn_error_string",
               "attn_version", "attn_debug_inject_fault", "attn_paged_append", "attn_decode_paged",
               "attn_decode_paged_workspace", "attn_key_weights", "attn_cache_evict",
               "attn_fwd_packed", "attn_fwd_packed_workspace", "attn_bwd_packed",
               "attn_bwd_packed_workspace", "attn_rope", "attn_rope_append",
               "attn_rope_frequencies", "attn_cache_plan")

_lib = None
_lock = threading.Lock()


class Rows(ctypes.Structure):
    """attn_rows_t: rows of heads at any strides, in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_longlong),
                ("row", ctypes.c_longlong), ("head", ctypes.c_longlong)]


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} ({code})")


def load():
    """Load (once) and return the ctypes handle of the built library."""
    global _lib
    if _lib is not None:   # (set once everything about it is)
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
            lib = ctypes.CDLL(LIB_PATH)
            vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            lib.attn_fwd.restype = i
            lib.attn_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
            lib.attn_fwd_lse.restype = i
            lib.attn_fwd_lse.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
            lib.attn_bwd.restype = i
            lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
            lib.attn_fwd_chunk.restype = i
            lib.attn_fwd_chunk.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp]
            lib.attn_decode.restype = i
            lib.attn_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
            lib.attn_decode_ring.restype = i
            lib.attn_decode_ring.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
            lib.attn_decode_noalloc.restype = i
            lib.attn_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
            lib.attn_paged_append.restype = i
            lib.attn_paged_append.argtypes = [vp] * 7 + [i] * 7 + [vp]
            lib.attn_decode_paged.restype = i
            lib.attn_decode_paged.argtypes = ([vp] * 7 + [i, i, vp, ctypes.c_size_t] + [i] * 8
                                              + [f, vp])
            lib.attn_decode_paged_workspace.restype = i
            lib.attn_decode_paged_workspace.argtypes = [i] * 7 + [ctypes.POINTER(ctypes.c_size_t)]
            lib.attn_key_weights.restype = i
            lib.attn_key_weights.argtypes = [vp] * 5 + [i] * 10 + [f, vp]
            lib.attn_cache_evict.restype = i
            lib.attn_cache_evict.argtypes = [vp, vp, vp, i, vp, vp, i, i, vp, i, vp, i, vp, vp] \
                + [i] * 6 + [vp]
            size = ctypes.POINTER(ctypes.c_size_t)
            rows = ctypes.POINTER(Rows)
            lib.attn_fwd_packed.restype = i
            lib.attn_fwd_packed.argtypes = ([rows] * 4 + [vp, vp, vp, ctypes.c_size_t] + [i] * 7
                                            + [f, vp])
            lib.attn_fwd_packed_workspace.restype = i
            lib.attn_fwd_packed_workspace.argtypes = [i] * 5 + [size]
            lib.attn_bwd_packed.restype = i
            lib.attn_bwd_packed.argtypes = ([rows] * 5 + [vp] + [rows] * 3
                                            + [vp, vp, ctypes.c_size_t] + [i] * 7 + [f, vp])
            lib.attn_bwd_packed_workspace.restype = i
            lib.attn_bwd_packed_workspace.argtypes = [i, i, i, size]
            lib.attn_rope.restype = i
            lib.attn_rope.argtypes = [rows, rows, i, rows, rows, i, vp, vp, f] + [i] * 6 + [vp]
            lib.attn_rope_append.restype = i
            lib.attn_rope_append.argtypes = ([rows, rows, i, rows, rows, rows, i, vp, vp, f, vp, vp,
                                              vp] + [i] * 7 + [vp])
            lib.attn_rope_frequencies.restype = i
            lib.attn_rope_frequencies.argtypes = [vp, vp, i, ctypes.c_double, i] \
                + [ctypes.c_double] * 4
            lib.attn_cache_plan.restype = i
            lib.attn_cache_plan.argtypes = [vp] * 10 + [i] * 6 + [vp]
            lib.attn_status.restype = i
            lib.attn_status.argtypes = [vp]
            lib.attn_error_string.restype = ctypes.c_char_p
            lib.attn_error_string.argtypes = [i]
            lib.attn_version.restype = i
            lib.attn_version.argtypes = []
            lib.attn_debug_inject_fault.restype = i
            lib.attn_debug_inject_fault.argtypes = [i]
            _lib = lib
    return _lib


def error_string(code: int) -> str:
    return load().attn_error_string(int(code)).decode()


def version() -> int:
    return int(load().attn_version())


# The current stream's handle without building a torch.cuda.Stream object
# (torch.cuda.current_stream() costs about 3 us per call, a quarter of the
# host's time per library call); the public route where these are missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_handle(stream) -> int:
    if stream is None:
        if _raw_stream is not None and _current_device is not None:
            return int(_raw_stream(_current_device()))
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _check_bf16(name, t, ndim):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor")


def attn_fwd(q, k, v, o=None, *, causal=True, window=0, scale=0.0, stream=None):
    """O = softmax(Q K^T * scale + M) V.  q [B,Hq,S,Dh], k/v [B,Hkv,S,Dh] bf16.
    scale 0 means 1/sqrt(Dh).  Returns o (allocated if not given)."""
    _check_bf16("q", q, 4)
    _check_bf16("k", k, 4)
    _check_bf16("v", v, 4)
    B, Hq, S, Dh = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, S, Dh) or tuple(v.shape) != (B, Hkv, S, Dh):
        raise ValueError("k and v must be [B, Hkv, S, Dh] matching q")
    if o is None:
        o = torch.empty_like(q)
    else:
        _check_bf16("o", o, 4)
        if o.shape != q.shape:
            raise ValueError("o must have q's shape")
    rc = load().attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, Hq, Hkv, S,
                         Dh, int(bool(causal)), int(window), float(scale), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd")
    return o


def attn_fwd_lse(q, k, v, o=None, lse=None, *, causal=True, window=0, scale=0.0, stream=None):
    """attn_fwd that also returns each row's log-sum-exp lse [B,Hq,S] fp32
    (natural log of the softmax normaliser).  Returns (o, lse)."""
    _check_bf16("q", q, 4)
    _check_bf16("k", k, 4)
    _check_bf16("v", v, 4)
    B, Hq, S, Dh = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, S, Dh) or tuple(v.shape) != (B, Hkv, S, Dh):
        raise ValueError("k and v must be [B, Hkv, S, Dh] matching q")
    if o is None:
        o = torch.empty_like(q)
    else:
        _check_bf16("o", o, 4)
        if o.shape != q.shape:
            raise ValueError("o must have q's shape")
    if lse is None:
        lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    elif (lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, S) or not lse.is_cuda
          or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous CUDA float32 [B, Hq, S] tensor")
    rc = load().attn_fwd_lse(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                             lse.data_ptr(), B, Hq, Hkv, S, Dh, int(bool(causal)), int(window),
                             float(scale), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_lse")
    return o, lse


def attn_bwd(q, k, v, o, dout, lse, dq=None, dk=None, dv=None, *, causal=True, window=0,
             scale=0.0, stream=None):
    """Backward pass of attn_fwd_lse: (dq, dk, dv) from q, k, v, its output o,
    its lse and dout = dL/do (all as attn_fwd_lse took / returned them)."""
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_bf16(name, t, 4)
    B, Hq, S, Dh = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, S, Dh) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, S, Dh] matching q")
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must have q's shape")
    if (lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, S) or not lse.is_cuda
            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous CUDA float32 [B, Hq, S] tensor")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t, ref in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        _check_bf16(name, t, 4)
        if t.shape != ref.shape:
            raise ValueError(f"{name} must have the shape of its input")
    rc = load().attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                         lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv,
                         S, Dh, int(bool(causal)), int(window), float(scale),
                         _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd")
    return dq, dk, dv


def attn_fwd_chunk(q, kcache, vcache, start_pos, o=None, *, causal=True, window=0, scale=0.0,
                   stream=None):
    """Prefill of one chunk against a KV cache.  q [B,Hq,Sq,Dh]; caches
    [B,Hkv,Tmax,Dh] bf16 already holding the chunk's keys/values at rows
    start_pos .. start_pos+Sq-1.  Query row r sits at position start_pos + r."""
    _check_bf16("q", q, 4)
    _check_bf16("kcache", kcache, 4)
    _check_bf16("vcache", vcache, 4)
    B, Hq, Sq, Dh = q.shape
    Hkv, Tmax = kcache.shape[1], kcache.shape[2]
    if tuple(kcache.shape) != (B, Hkv, Tmax, Dh) or vcache.shape != kcache.shape:
        raise ValueError("the caches must be [B, Hkv, Tmax, Dh] matching q")
    if o is None:
        o = torch.empty_like(q)
    else:
        _check_bf16("o", o, 4)
        if o.shape != q.shape:
            raise ValueError("o must have q's shape")
    rc = load().attn_fwd_chunk(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(), o.data_ptr(), B,
                               Hq, Hkv, Sq, Tmax, int(start_pos), Dh, int(bool(causal)),
                               int(window), float(scale), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_chunk")
    return o


def attn_decode(q, kcache, vcache, seqlens, o=None, *, window=0, scale=0.0, stream=None):
    """One decode step.  q [B,Hq,1,Dh]; caches [B,Hkv,Tmax,Dh] bf16; seqlens
    [B] int32 on the device (keys held per sequence, own key included)."""
    _check_bf16("q", q, 4)
    _check_bf16("kcache", kcache, 4)
    _check_bf16("vcache", vcache, 4)
    B, Hq, one, Dh = q.shape
    Hkv, Tmax = kcache.shape[1], kcache.shape[2]
    if one != 1 or tuple(kcache.shape) != (B, Hkv, Tmax, Dh) or vcache.shape != kcache.shape:
        raise ValueError("q must be [B,Hq,1,Dh] and the caches [B,Hkv,Tmax,Dh]")
    if (not isinstance(seqlens, torch.Tensor) or seqlens.dtype != torch.int32 or not seqlens.is_cuda
            or seqlens.numel() != B or not seqlens.is_contiguous()):
        raise TypeError("seqlens must be a contiguous CUDA int32 tensor of B entries")
    if o is None:
        o = torch.empty_like(q)
    else:
        _check_bf16("o", o, 4)
        if o.shape != q.shape:
            raise ValueError("o must have q's shape")
    rc = load().attn_decode(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(), seqlens.data_ptr(),
                            o.data_ptr(), B, Hq, Hkv, Tmax, Dh, int(window), float(scale),
                            _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode")
    return o


def attn_decode_ring(q, kcache, vcache, seqlens, o=None, *, window=0, scale=0.0, stream=None):
    """Decode step over a rolling-buffer cache [B,Hkv,C,Dh]: position t of
    sequence b at row t % C; seqlens [B] int32 = tokens so far (see
    include/attn.h)."""
    _check_bf16("q", q, 4)
    _check_bf16("kcache", kcache, 4)
    _check_bf16("vcache", vcache, 4)
    B, Hq, one, Dh = q.shape
    Hkv, C = kcache.shape[1], kcache.shape[2]
    if one != 1 or tuple(kcache.shape) != (B, Hkv, C, Dh) or vcache.shape != kcache.shape:
        raise ValueError("q must be [B,Hq,1,Dh] and the caches [B,Hkv,C,Dh]")
    if (not isinstance(seqlens, torch.Tensor) or seqlens.dtype != torch.int32 or not seqlens.is_cuda
            or seqlens.numel() != B or not seqlens.is_contiguous()):
        raise TypeError("seqlens must be a contiguous CUDA int32 tensor of B entries")
    if o is None:
        o = torch.empty_like(q)
    else:
        _check_bf16("o", o, 4)
        if o.shape != q.shape:
            raise ValueError("o must have q's shape")
    rc = load().attn_decode_ring(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(),
                                 seqlens.data_ptr(), o.data_ptr(), B, Hq, Hkv, C, Dh, int(window),
                                 float(scale), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_ring")
    return o


def attn_decode_noalloc(q, kcache, vcache, seqlens, o=None, *, window=0, scale=0.0,
                        stream=None):
    """attn_decode for callers that must not allocate device memory: the
    library's scratch is a fixed 16 MiB device array (see include/attn.h).
    Only the output, when not given, is allocated here by torch."""
    _check_bf16("q", q, 4)
    _check_bf16("kcache", kcache, 4)
    _check_bf16("vcache", vcache, 4)
    B, Hq, one, Dh = q.shape
    Hkv, Tmax = kcache.shape[1], kcache.shape[2]
    if one != 1 or tuple(kcache.shape) != (B, Hkv, Tmax, Dh) or vcache.shape != kcache.shape:
        raise ValueError("q must be [B,Hq,1,Dh] and the caches [B,Hkv,Tmax,Dh]")
    if (not isinstance(seqlens, torch.Tensor) or seqlens.dtype != torch.int32 or not seqlens.is_cuda
            or seqlens.numel() != B or not seqlens.is_contiguous()):
        raise TypeError("seqlens must be a contiguous CUDA int32 tensor of B entries")
    if o is None:
        o = torch.empty_like(q)
    else:
        _check_bf16("o", o, 4)
        if o.shape != q.shape:
            raise ValueError("o must have q's shape")
    rc = load().attn_decode_noalloc(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(),
                                    seqlens.data_ptr(), o.data_ptr(), B, Hq, Hkv, Tmax, Dh,
                                    int(window), float(scale), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_noalloc")
    return o


def attn_debug_inject_fault(kind: int) -> None:
    """Test hook (see include/attn.h): 0 none, 1 a prefill K tile is withheld,
    2 a decode key block (CUDA-core path), 3 a decode K tile (tensor-core path);
    later launches wait, give up and report ATTN_ERR_TIMEOUT through attn_status()."""
    rc = load().attn_debug_inject_fault(int(kind))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_debug_inject_fault")


def attn_status(stream=None) -> int:
    """Synchronise the stream; return and clear the device's latched error code."""
    return int(load().attn_status(_stream_handle(stream)))


# ---------------------------------------------------------------------------
# the paged cache (include/attn.h)

def _this_device() -> int:
    return _current_device() if _current_device is not None else torch.cuda.current_device()


def _check(name, t, dtype, shape, device):
    """A contiguous tensor of that type and shape, on the same GPU as the others."""
    try:   # (most of a small call's time is checks: isinstance on a Tensor is not cheap)
        if (t.dtype is dtype and t.shape == shape and t.get_device() == device >= 0
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor, got {list(t.shape)}")
    raise ValueError(f"{name} must be on the same device as the other tensors")


def _check_current(device):
    """The library launches on the current device (a stream belongs to one)."""
    if device != _this_device():
        raise ValueError("the tensors must be on the current device (torch.cuda.device)")


def _shape(name, t, ndim):
    """The shape of a tensor of ndim axes."""
    shape = getattr(t, "shape", None)
    if shape is None:
        raise TypeError(f"{name} must be a tensor")
    if len(shape) != ndim:
        raise ValueError(f"{name} must have {ndim} axes")
    return shape


def _int32(name, x):
    """An int that the library takes: a larger one would lose its upper bits."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} must fit in 32 bits")
    return x


def _check_pools(kpages, vpages, table, seqlens):
    """The checks that every paged call makes: (B, Hkv, num_pages, page, cols, Dh, device)."""
    P, Hkv, page, Dh = shape = _shape("kpages", kpages, 4)
    B, cols = table_shape = _shape("table", table, 2)
    if B > 0x7fffffff or cols > 0x7fffffff:
        raise ValueError("table must have less than 2^31 entries along each axis")
    device = kpages.get_device()
    _check("kpages", kpages, torch.bfloat16, shape, device)
    _check_current(device)
    _check("vpages", vpages, torch.bfloat16, shape, device)
    _check("table", table, torch.int32, table_shape, device)
    _check("seqlens", seqlens, torch.int32, (B,), device)
    return B, Hkv, P, page, cols, Dh, device


def _rows_of(name, t, B, Hkv, device):
    """A contiguous float32 [B, Hkv, stride] tensor: its stride."""
    stride = _shape(name, t, 3)[2]
    if stride > 0x7fffffff:
        raise ValueError(f"{name} must have less than 2^31 entries per row")
    _check(name, t, torch.float32, (B, Hkv, stride), device)
    return stride


def _empty(shape, dtype, device, stream):
    """A tensor whose memory belongs to the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def attn_paged_append(k, v, kpages, vpages, table, seqlens, newlens=None, *, stream=None):
    """Write new keys and values k, v [B,Hkv,S,Dh] to a paged cache: pools
    [P,Hkv,page,Dh] bf16, table [B,cols] int32, seqlens [B] int32 = keys held
    after the append, newlens [B] int32 = real rows of k and v (None: all S).
    Returns (kpages, vpages), which are written in place."""
    B, Hkv, P, page, cols, Dh, device = _check_pools(kpages, vpages, table, seqlens)
    S = _shape("k", k, 4)[2]
    _check("k", k, torch.bfloat16, (B, Hkv, S, Dh), device)
    _check("v", v, torch.bfloat16, (B, Hkv, S, Dh), device)
    if newlens is not None:
        _check("newlens", newlens, torch.int32, (B,), device)
    rc = load().attn_paged_append(k.data_ptr(), v.data_ptr(), kpages.data_ptr(), vpages.data_ptr(),
                                  table.data_ptr(), seqlens.data_ptr(),
                                  None if newlens is None else newlens.data_ptr(), B, Hkv, S, P,
                                  page, cols, Dh, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_paged_append")
    return kpages, vpages


@functools.lru_cache(maxsize=4096)
def _decode_paged_workspace(device, B, Hq, Hkv, page, cols, Dh, with_weights):
    size = ctypes.c_size_t()
    rc = load().attn_decode_paged_workspace(B, Hq, Hkv, page, cols, Dh, int(with_weights),
                                            ctypes.byref(size))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_paged_workspace")
    return size.value


def attn_decode_paged_workspace(q, kpages, table, *, weights=False):
    """Bytes of workspace that attn_decode_paged needs on the current device for
    tensors of these shapes, with or without weights."""
    B, Hq, one, Dh = _shape("q", q, 4)
    _, Hkv, page, cache_Dh = _shape("kpages", kpages, 4)
    table_B, cols = _shape("table", table, 2)
    if one != 1 or cache_Dh != Dh or table_B != B:
        raise ValueError("q must be [B,Hq,1,Dh], kpages [P,Hkv,page,Dh] and table [B,cols]")
    for name, x in (("q", max(B, Hq, Dh)), ("kpages", max(Hkv, page)), ("table", cols)):
        if x > 0x7fffffff:
            raise ValueError(f"{name} must have less than 2^31 entries along each axis")
    return _decode_paged_workspace(_this_device(), B, Hq, Hkv, page, cols, Dh, bool(weights))


def attn_decode_paged(q, kpages, vpages, table, seqlens, o=None, *, window=0, scale=0.0,
                      weights=None, accumulate=True, workspace=None, stream=None):
    """One decode step over a paged cache (see attn_paged_append).  q
    [B,Hq,1,Dh]; a length of 0 gives a zero output.  Where the softmax weights
    meet V they are rounded to bf16, or with up to 16 query heads per K/V head
    held to two parts of it.  weights [B,Hkv,rows] fp32 (rows >= cols * page)
    receives each key's softmax weight summed over its query heads, added to
    what is there or, with accumulate=False, in its place.  workspace: a uint8
    tensor of attn_decode_paged_workspace() bytes (None: allocated here by
    torch, on the call's stream).  Returns o."""
    window = _int32("window", window)
    B, Hkv, P, page, cols, Dh, device = _check_pools(kpages, vpages, table, seqlens)
    Hq = _shape("q", q, 4)[1]
    _check("q", q, torch.bfloat16, (B, Hq, 1, Dh), device)
    stride = 0 if weights is None else _rows_of("weights", weights, B, Hkv, device)
    need = _decode_paged_workspace(device, B, Hq, Hkv, page, cols, Dh, weights is not None)
    if o is not None:
        _check("o", o, torch.bfloat16, (B, Hq, 1, Dh), device)
    if workspace is not None and (not isinstance(workspace, torch.Tensor)
                                  or workspace.dtype != torch.uint8
                                  or workspace.get_device() != device
                                  or not workspace.is_contiguous()):
        raise TypeError("workspace must be a contiguous CUDA uint8 tensor on the same device")
    if o is None:
        o = _empty((B, Hq, 1, Dh), torch.bfloat16, q.device, stream)
    if workspace is None and need > 0:
        workspace = _empty((need,), torch.uint8, q.device, stream)
    rc = load().attn_decode_paged(q.data_ptr(), kpages.data_ptr(), vpages.data_ptr(),
                                  table.data_ptr(), seqlens.data_ptr(), o.data_ptr(),
                                  None if weights is None else weights.data_ptr(), stride,
                                  int(bool(accumulate)),
                                  None if workspace is None else workspace.data_ptr(),
                                  0 if workspace is None else workspace.numel(),
                                  B, Hq, Hkv, P, page, cols, Dh, window, float(scale),
                                  _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_paged")
    return o


def attn_key_weights(q, k, lse, weights, seqlens=None, *, queries=0, causal=True, window=0,
                     scale=0.0, accumulate=True, stream=None):
    """The softmax weight that each key of a prompt received, summed over the
    query heads of its K/V head and over the last `queries` queries (0: all):
    weights [B,Hkv,rows] fp32, rows >= S, is added to, or replaced with
    accumulate=False.  q [B,Hq,S,Dh], k [B,Hkv,S,Dh] and lse [B,Hq,S] as
    attn_fwd_lse took and returned them; seqlens [B] int32: the real rows of a
    padded prompt.  Returns weights."""
    queries, window = _int32("queries", queries), _int32("window", window)
    B, Hq, S, Dh = shape = _shape("q", q, 4)
    Hkv = _shape("k", k, 4)[1]
    device = q.get_device()
    _check("q", q, torch.bfloat16, shape, device)
    _check_current(device)
    _check("k", k, torch.bfloat16, (B, Hkv, S, Dh), device)
    _check("lse", lse, torch.float32, (B, Hq, S), device)
    stride = _rows_of("weights", weights, B, Hkv, device)
    if seqlens is not None:
        _check("seqlens", seqlens, torch.int32, (B,), device)
    rc = load().attn_key_weights(q.data_ptr(), k.data_ptr(), lse.data_ptr(),
                                 None if seqlens is None else seqlens.data_ptr(),
                                 weights.data_ptr(), stride, B, Hq, Hkv, S, Dh, queries,
                                 int(bool(causal)), window, int(bool(accumulate)),
                                 float(scale), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_key_weights")
    return weights


def attn_cache_evict(kpages, vpages, weights, table, seqlens, budget, recent=0, *, table_out=None,
                     weights_out=None, newlens=None, keep=None, stream=None):
    """Shrink each sequence of a paged cache to at most `budget` keys: the last
    `recent` rows and those with the largest weights [B,Hkv,rows] fp32 before
    them, per K/V head, in their order.  The kept rows move to the pages of
    table_out [B,cols_out] int32 (None: in place), their weights to
    weights_out (None: in place).  Returns (newlens [B], keep [B,Hkv,budget]):
    the new lengths, and each kept row's former number (then -1)."""
    budget, recent = _int32("budget", budget), _int32("recent", recent)
    B, Hkv, P, page, cols, Dh, device = _check_pools(kpages, vpages, table, seqlens)
    stride = _rows_of("weights", weights, B, Hkv, device)
    cols_out, stride_out = cols, stride
    if table_out is not None:
        cols_out = _shape("table_out", table_out, 2)[1]
        _check("table_out", table_out, torch.int32, (B, cols_out), device)
    if weights_out is not None:
        stride_out = _rows_of("weights_out", weights_out, B, Hkv, device)
    if budget < 1:
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_cache_evict")
    if newlens is not None:
        _check("newlens", newlens, torch.int32, (B,), device)
    if keep is not None:
        _check("keep", keep, torch.int32, (B, Hkv, budget), device)
    if newlens is None:
        newlens = _empty((B,), torch.int32, seqlens.device, stream)
    if keep is None:
        keep = _empty((B, Hkv, budget), torch.int32, seqlens.device, stream)
    rc = load().attn_cache_evict(kpages.data_ptr(), vpages.data_ptr(), weights.data_ptr(), stride,
                                 table.data_ptr(), seqlens.data_ptr(), budget, recent,
                                 None if table_out is None else table_out.data_ptr(), cols_out,
                                 None if weights_out is None else weights_out.data_ptr(),
                                 stride_out, newlens.data_ptr(), keep.data_ptr(), B, Hkv, P, page,
                                 cols, Dh, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_cache_evict")
    return newlens, keep


# ---------------------------------------------------------------------------
# packed sequences, rotary positions, the plan of a serving step (include/attn.h)

def _heads(name, t, shape, device):
    """A bf16 tensor of that shape, [T, H, Dh] or a batch [B, H, S, Dh], on that GPU, the values
    of a head side by side: as the library takes it."""
    try:
        stride = t.stride()
        if (t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == device >= 0
                and stride[-1] == 1):
            if len(stride) == 3:
                return Rows(t.data_ptr(), 0, stride[0], stride[1])
            return Rows(t.data_ptr(), stride[0], stride[2], stride[1])
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"the values of a head must lie side by side in {name}")
    raise ValueError(f"{name} must be on the same device as the other tensors")


_MOST = 0x7fffffff


def _packed_shape(q, k, cu_seqlens):
    """B, Hq, Hkv, T, Dh and device of a packed call."""
    T, Hq, Dh = _shape("q", q, 3)
    Hkv = _shape("k", k, 3)[1]
    n, = _shape("cu_seqlens", cu_seqlens, 1)
    if n < 1 or n > _MOST or T > _MOST or Hq > _MOST:
        raise ValueError("cu_seqlens must have B + 1 entries, and less than 2^31 rows and heads")
    device = q.get_device()
    if device < 0:
        raise TypeError("q must be a CUDA bfloat16 tensor")
    _check_current(device)
    _check("cu_seqlens", cu_seqlens, torch.int32, (n,), device)
    return n - 1, Hq, Hkv, T, Dh, device


@functools.lru_cache(maxsize=4096)
def _packed_workspace(device, B, Hq, T, Dh, causal, backward):
    size = ctypes.c_size_t()
    if backward:
        rc = load().attn_bwd_packed_workspace(B, Hq, T, ctypes.byref(size))
    else:
        rc = load().attn_fwd_packed_workspace(B, Hq, T, Dh, causal, ctypes.byref(size))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_packed_workspace" if backward else "attn_fwd_packed_workspace")
    return size.value


def attn_packed_workspace(q, cu_seqlens, *, causal=True, backward=False):
    """Bytes of workspace that attn_fwd_packed, or attn_bwd_packed, needs on the
    current device for tensors of these shapes."""
    T, Hq, Dh = _shape("q", q, 3)
    n = _shape("cu_seqlens", cu_seqlens, 1)[0]
    return _packed_workspace(_this_device(), _int32("the number of sequences", n - 1),
                             _int32("heads", Hq), _int32("rows", T), _int32("values", Dh),
                             int(bool(causal)), bool(backward))


def _workspace(workspace, need, device, tensor, stream):
    """The workspace's address and size (and the tensor, which the caller keeps)."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _empty((need,), torch.uint8, tensor.device, stream)
        return workspace.data_ptr(), need, workspace
    if (not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8
            or workspace.get_device() != device or not workspace.is_contiguous()):
        raise TypeError("workspace must be a contiguous CUDA uint8 tensor on the same device")
    return workspace.data_ptr(), workspace.numel(), workspace


def attn_fwd_packed(q, k, v, cu_seqlens, o=None, lse=None, *, causal=True, window=0, scale=0.0,
                    workspace=None, stream=None):
    """attn_fwd of sequences that lie one behind another: q [T,Hq,Dh], k and v
    [T,Hkv,Dh] bf16 at any strides (slices of one projection's output as they
    are), cu_seqlens [B+1] int32 the first row of each sequence and the last
    one's end.  lse [Hq,T] fp32, where given, receives the log-sum-exps.  Rows
    of no sequence keep what o and lse hold (nothing, where o is allocated
    here).  workspace: a uint8 tensor of attn_packed_workspace() bytes (None:
    allocated here by torch, on the call's stream, where any is needed).
    Returns o."""
    window, causal = _int32("window", window), 1 if causal else 0
    B, Hq, Hkv, T, Dh, device = _packed_shape(q, k, cu_seqlens)
    rq = _heads("q", q, (T, Hq, Dh), device)
    rk = _heads("k", k, (T, Hkv, Dh), device)
    rv = _heads("v", v, (T, Hkv, Dh), device)
    if lse is not None:
        _check("lse", lse, torch.float32, (Hq, T), device)
    if o is None:
        o = _empty((T, Hq, Dh), torch.bfloat16, q.device, stream)
    ro = _heads("o", o, (T, Hq, Dh), device)
    ws, size, keep = _workspace(workspace,
                                _packed_workspace(device, B, Hq, T, Dh, causal, False), device, q,
                                stream)
    rc = load().attn_fwd_packed(rq, rk, rv, ro, None if lse is None else lse.data_ptr(),
                                cu_seqlens.data_ptr(), ws, size, B, Hq, Hkv, T, Dh, causal, window,
                                float(scale), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_packed")
    return o


def attn_bwd_packed(q, k, v, o, dout, lse, cu_seqlens, dq=None, dk=None, dv=None, *, causal=True,
                    window=0, scale=0.0, workspace=None, stream=None):
    """Backward pass of attn_fwd_packed: (dq, dk, dv) from its inputs, the o and
    lse [Hq,T] it gave for them (not ones joined from several sets of keys:
    queries of few keys take nothing from o), and dout = dL/do.  The gradients
    may be slices of one wider tensor, as q, k and v may; rows of no sequence
    are not written."""
    window = _int32("window", window)
    B, Hq, Hkv, T, Dh, device = _packed_shape(q, k, cu_seqlens)
    wide, narrow = (T, Hq, Dh), (T, Hkv, Dh)
    _check("lse", lse, torch.float32, (Hq, T), device)
    ins = [_heads(name, t, shape, device) for name, t, shape in (
        ("q", q, wide), ("k", k, narrow), ("v", v, narrow), ("o", o, wide), ("dout", dout, wide))]
    dq = _empty(wide, torch.bfloat16, q.device, stream) if dq is None else dq
    dk = _empty(narrow, torch.bfloat16, q.device, stream) if dk is None else dk
    dv = _empty(narrow, torch.bfloat16, q.device, stream) if dv is None else dv
    outs = [_heads(name, t, shape, device) for name, t, shape in (
        ("dq", dq, wide), ("dk", dk, narrow), ("dv", dv, narrow))]
    ws, size, keep = _workspace(workspace, _packed_workspace(device, B, Hq, T, Dh, 1, True), device,
                                q, stream)
    rc = load().attn_bwd_packed(*ins, lse.data_ptr(), *outs, cu_seqlens.data_ptr(), ws,
                                size, B, Hq, Hkv, T, Dh, int(bool(causal)), window, float(scale),
                                _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_packed")
    return dq, dk, dv


class RopeFrequencies(typing.NamedTuple):
    """turns [rotary_dim/2] int64 on the GPU (2^-64 turns per token) and the
    factor on the turned values."""
    turns: torch.Tensor
    amplitude: float


_SCALINGS = {"none": 0, "linear": 1, "base": 2, "turns": 3, "yarn": 4}


def attn_rope_frequencies(rotary_dim, base=10000.0, *, scaling="none", factor=1.0, low=1.0,
                          high=None, original_len=8192, device="cuda"):
    """What attn_rope turns by: base^(-2 i / rotary_dim) radians per token for
    pair i, scaled for a longer context by "linear", "base", "turns" (pairs by
    the turns they make over original_len: kept from `high` on, divided by
    factor up to `low`, blended between; high is 4) or "yarn" (the same with an
    amplitude, high 32).  Both blend linearly in the turns, as YaRN was
    published; models whose own code blends linearly in the pair's number have
    other frequencies, which a RopeFrequencies takes as they are.  See
    include/attn.h."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    rotary_dim = _int32("rotary_dim", rotary_dim)
    turns = torch.zeros(max(rotary_dim // 2, 1), dtype=torch.int64)
    amplitude = ctypes.c_float()
    rc = load().attn_rope_frequencies(turns.data_ptr() if 0 < rotary_dim <= 256 else None,
                                      ctypes.addressof(amplitude), rotary_dim, float(base),
                                      _SCALINGS[scaling], float(factor), float(low), float(high),
                                      float(original_len))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope_frequencies")
    return RopeFrequencies(turns.to(device), amplitude.value)


def _rope_shape(q, k, positions, turns):
    """What both rotations check: B, S, Hq, Hkv, Dh, rotary_dim, device and the shapes."""
    shape = getattr(q, "shape", ())
    axes = len(shape)
    if axes == 3:
        S, Hq, Dh = shape
        Hkv = _shape("k", k, 3)[1]
        B, kshape, pshape = 1, (S, Hkv, Dh), (S,)
    elif axes == 4:
        B, Hq, S, Dh = shape
        Hkv = _shape("k", k, 4)[1]
        kshape, pshape = (B, Hkv, S, Dh), (B, S)
    else:
        raise ValueError("q must be [T,Hq,Dh] or [B,Hq,S,Dh]")
    if S > _MOST or B > _MOST or Hq > _MOST or Hkv > _MOST:
        raise ValueError("q and k must have less than 2^31 entries along each axis")
    device = q.get_device()
    if device < 0:
        raise TypeError("q must be a CUDA bfloat16 tensor")
    _check_current(device)
    _check("positions", positions, torch.int32, pshape, device)
    n, = _shape("turns", turns, 1)
    _check("turns", turns, torch.int64, (n,), device)
    return B, S, Hq, Hkv, Dh, 2 * n, device, shape, kshape


def attn_rope(q, k, positions, frequencies, q_out=None, k_out=None, *, interleaved=False,
              inverse=False, stream=None):
    """Rotary positions: the first rotary_dim values of each head of q and k,
    packed [T,H,Dh] or batches [B,H,S,Dh] at any strides, turned in pairs
    (halves, or with interleaved=True neighbours) by positions [T] or [B,S]
    int32 times `frequencies` (attn_rope_frequencies).  A negative position
    leaves the row out.  q_out and k_out may be q and k (in place); None:
    allocated here.  inverse=True turns the other way: the gradients of q and
    k from those of the outputs.  Returns (q_out, k_out)."""
    turns, amplitude = frequencies
    B, S, Hq, Hkv, Dh, rot, device, qs, ks = _rope_shape(q, k, positions, turns)
    rq, rk = _heads("q", q, qs, device), _heads("k", k, ks, device)
    if q_out is None:
        q_out = _empty(qs, torch.bfloat16, q.device, stream)
    if k_out is None:
        k_out = _empty(ks, torch.bfloat16, q.device, stream)
    rc = load().attn_rope(rq, _heads("q_out", q_out, qs, device), Hq, rk,
                          _heads("k_out", k_out, ks, device), Hkv, positions.data_ptr(),
                          turns.data_ptr(), amplitude, B, S, Dh, rot, 1 if interleaved else 0,
                          1 if inverse else 0, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope")
    return q_out, k_out


def attn_rope_append(q, k, v, positions, frequencies, kpages, vpages, slots, q_out=None,
                     k_out=None, *, interleaved=False, stream=None):
    """attn_rope of q and k, and the write of the turned k and of v to a paged
    cache (pools [P,Hkv,page,Dh]) in the same pass: slots [T] or [B,S] int32
    (attn_cache_plan gives them), a negative one writes nothing there.  q_out
    None: in place.  k_out None: the turned keys go to the cache alone.  Returns
    (q_out, k_out)."""
    turns, amplitude = frequencies
    B, S, Hq, Hkv, Dh, rot, device, qs, ks = _rope_shape(q, k, positions, turns)
    P, pool_heads, page, pool_Dh = pools = _shape("kpages", kpages, 4)
    if pool_heads != Hkv or pool_Dh != Dh or P > _MOST or page > _MOST:
        raise ValueError("kpages must be [P, Hkv, page, Dh] matching k")
    _check("kpages", kpages, torch.bfloat16, pools, device)
    _check("vpages", vpages, torch.bfloat16, pools, device)
    _check("slots", slots, torch.int32, positions.shape, device)
    rq, rk, rv = (_heads("q", q, qs, device), _heads("k", k, ks, device),
                  _heads("v", v, ks, device))
    if q_out is None:
        q_out, rqo = q, rq
    else:
        rqo = _heads("q_out", q_out, qs, device)
    rko = None if k_out is None else _heads("k_out", k_out, ks, device)
    rc = load().attn_rope_append(rq, rqo, Hq, rk, rko, rv, Hkv, positions.data_ptr(),
                                 turns.data_ptr(), amplitude, kpages.data_ptr(),
                                 vpages.data_ptr(), slots.data_ptr(), P, page, B, S, Dh, rot,
                                 1 if interleaved else 0, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope_append")
    return q_out, k_out


def attn_cache_plan(delta, seqlens, table, free_pages, num_free, *, rows, page, num_pages,
                    seqlens_out=None, num_free_out=None, cu_seqlens=None, positions=None,
                    slots=None, stream=None):
    """The pages, slots and positions of a serving step, from the lengths on the
    GPU: sequence b of a paged cache (table [B,cols], seqlens [B]) changes by
    delta[b] rows, new tokens or (negative) rows taken back.  Free pages are a
    stack: the first num_free [1] entries of free_pages.  Pages given back go
    onto it, then pages that new rows need come off it, into table.  Lengths
    and num_free change in place (or go to seqlens_out, num_free_out).  Returns
    (cu_seqlens [B+1], positions [rows], slots [rows]) of the packed new tokens,
    -1 behind the last (cu_seqlens[B] of them, the first `rows` of which have
    their place here); where pages do not suffice, nothing changes and
    attn_status() says so.  All int32."""
    rows, page, num_pages = (_int32("rows", rows), _int32("page", page),
                             _int32("num_pages", num_pages))
    B, cols = shape = _shape("table", table, 2)
    capacity, = _shape("free_pages", free_pages, 1)
    if B > _MOST or cols > _MOST or capacity > _MOST:
        raise ValueError("table and free_pages must have less than 2^31 entries along each axis")
    if rows < 0:
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_cache_plan")
    device = table.get_device()
    int32, batch, one = torch.int32, (B,), (1,)
    _check("table", table, int32, shape, device)
    _check_current(device)
    _check("delta", delta, int32, batch, device)
    _check("seqlens", seqlens, int32, batch, device)
    _check("free_pages", free_pages, int32, (capacity,), device)
    _check("num_free", num_free, int32, one, device)
    if seqlens_out is None:
        seqlens_out = seqlens
    else:
        _check("seqlens_out", seqlens_out, int32, batch, device)
    if num_free_out is None:
        num_free_out = num_free
    else:
        _check("num_free_out", num_free_out, int32, one, device)
    if cu_seqlens is None:
        cu_seqlens = _empty((B + 1,), int32, table.device, stream)
    else:
        _check("cu_seqlens", cu_seqlens, int32, (B + 1,), device)
    if positions is None:
        positions = _empty((rows,), int32, table.device, stream)
    else:
        _check("positions", positions, int32, (rows,), device)
    if slots is None:
        slots = _empty((rows,), int32, table.device, stream)
    else:
        _check("slots", slots, int32, (rows,), device)
    rc = load().attn_cache_plan(delta.data_ptr(), seqlens.data_ptr(), seqlens_out.data_ptr(),
                                table.data_ptr(), free_pages.data_ptr(), num_free.data_ptr(),
                                num_free_out.data_ptr(), cu_seqlens.data_ptr(),
                                positions.data_ptr(), slots.data_ptr(), B, cols, page, num_pages,
                                capacity, rows, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_cache_plan")
    return cu_seqlens, positions, slots
