"""Python binding of the 8-bit key/value cache of libmlora.so
(include/mlora_kv.h).  Argument marshalling only: every step runs in the
library's CUDA kernels; PyTorch provides device memory and streams.

    cache = KvCache.empty(n_pages, n_kv_heads, head_dim)     # or KvCache(k, v, k_scale, v_scale)
    ws = kv_workspace()
    kv_append(cache, page_table, kv_len, k, v)                              # newest rows into the cache
    out, lse = kv_attention(cache, page_table, kv_len, q, max_len, workspace=ws)
    k, v = kv_read(cache, page_table, kv_len, n_rows)                       # back as fp32 or bf16
    kv_check_status(cache)                                                  # 0, or -2 (E_RANGE)

Rollouts of the transformer model over one cache per layer:

    tf_forward_cached(h, caches, prompt, None, adapter_ids, page_table, kv_len, max_len, row_off, max_rows)
    token, logprob = tf_sample_cached(h, caches, token, adapter_ids, uniforms, page_table, kv_len, max_len)

page_table int32 [n_seqs, max_pages], kv_len int32 [n_seqs] (the lengths with
the call's rows counted) and row_off int32 [n_seqs + 1] (None: one row a
sequence) are CUDA tensors; max_rows and max_len are upper bounds the caller
knows on the host.
"""
from __future__ import annotations

import ctypes
import math
from ctypes import POINTER, byref, c_float, c_int32, c_int64, c_void_p

import torch

from . import _check, load_library
from .transformer import _TfBatch

__all__ = ["PAGE", "KvCache", "kv_workspace", "kv_append", "kv_read", "kv_attention", "kv_check_status",
           "tf_forward_cached", "tf_sample_cached"]

PAGE = 64
WORKSPACE_BYTES = 32 << 20


class _KvCache(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p),
                ("status", c_void_p), ("n_pages", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32)]


class _KvSeqs(ctypes.Structure):
    _fields_ = [("page_table", c_void_p), ("kv_len", c_void_p), ("row_off", c_void_p), ("n_rows", c_int64),
                ("n_seqs", c_int32), ("max_pages", c_int32), ("max_rows", c_int32)]


class _KvAttn(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("out", c_void_p), ("lse", c_void_p), ("workspace", c_void_p),
                ("q_stride", c_int64), ("out_stride", c_int64), ("workspace_bytes", c_int64), ("max_len", c_int64),
                ("dtype", c_int32), ("n_heads", c_int32), ("scale", c_float)]


class _TfContext(ctypes.Structure):
    _fields_ = [("caches", POINTER(_KvCache)), ("seqs", _KvSeqs), ("workspace", c_void_p),
                ("workspace_bytes", c_int64), ("max_len", c_int64)]


_SIGNATURES = {
    "mlora_kv_append": (c_int32, [POINTER(_KvCache), POINTER(_KvSeqs), c_int32, c_void_p, c_int64, c_void_p,
                                  c_int64, c_void_p]),
    "mlora_kv_read": (c_int32, [POINTER(_KvCache), POINTER(_KvSeqs), c_int32, c_void_p, c_void_p, c_void_p]),
    "mlora_kv_attention": (c_int32, [POINTER(_KvCache), POINTER(_KvSeqs), POINTER(_KvAttn), c_void_p]),
    "mlora_tf_forward_cached": (c_int32, [c_void_p, POINTER(_TfBatch), POINTER(_TfContext), c_void_p, c_void_p]),
    "mlora_tf_sample_cached": (c_int32, [c_void_p, POINTER(_TfBatch), POINTER(_TfContext), c_void_p, c_void_p,
                                         c_void_p, c_void_p]),
}

_kv_lib = None


def _lib():
    global _kv_lib
    if _kv_lib is None:
        lib = load_library()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _kv_lib = lib
    return _kv_lib


_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_INT32, _FLOAT32 = torch.int32, torch.float32


def _dtype(t) -> int:
    d = _DTYPES.get(t)
    if d is None:
        raise ValueError(f"dtype {t}: bfloat16 or float32 is needed")
    return d


def _on(index: int, stream) -> int:
    """The stream's handle (None: the current one of device `index`, which has to be the current device)."""
    if torch.cuda.current_device() != index:
        raise ValueError(f"the tensors are on cuda:{index}, which is not the current device")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A tensor whose memory belongs to the stream that will use it: blocks of another
    stream's pool can still be in use there, or be handed out again too early."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class KvCache:
    """A pool of cache pages: uint8 k, v [n_pages, n_kv_heads, 64, head_dim]
    (the byte order inside a tile is the library's) and float32 k_scale, v_scale
    [n_pages, n_kv_heads], contiguous CUDA tensors that the cache keeps alive."""

    def __init__(self, k, v, k_scale, v_scale):
        n_pages, n_kv, page, hd = k.shape
        if page != PAGE or tuple(v.shape) != tuple(k.shape):
            raise ValueError(f"k and v must be [n_pages, n_kv_heads, {PAGE}, head_dim]")
        for t, dt, shape in ((k, torch.uint8, k.shape), (v, torch.uint8, k.shape),
                             (k_scale, torch.float32, (n_pages, n_kv)), (v_scale, torch.float32, (n_pages, n_kv))):
            if t.dtype != dt or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != k.device:
                raise ValueError("cache tensors must be contiguous, on one device, uint8 pages and float32 scales")
        if not k.is_cuda:
            raise ValueError("cache tensors must be CUDA tensors")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self.n_pages, self.n_kv_heads, self.head_dim, self.device = n_pages, n_kv, hd, k.device
        self.index = k.get_device()
        self._c = _KvCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                           self.status.data_ptr(), n_pages, n_kv, hd)
        self._ref = byref(self._c)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, head_dim: int, device="cuda") -> "KvCache":
        shape = (n_pages, n_kv_heads, PAGE, head_dim)
        return cls(*[torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)],
                   *[torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2)])


def kv_workspace(device="cuda", nbytes: int = WORKSPACE_BYTES):
    """A workspace of kv_attention; calls that may overlap need one each.  With
    nbytes = 0 no sequence is cut and results do not depend on the batch."""
    return torch.empty(int(nbytes), dtype=torch.uint8, device=device)


def _ids(name, t, shape, index) -> int:
    if t.dtype is not _INT32 or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on the cache's device")
    return t.data_ptr()


def _out(name, t, n, index) -> int:
    if t.dtype is not _FLOAT32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous float32 tensor [{n}] on the cache's device")
    return t.data_ptr()


def _seqs(cache, page_table, kv_len, row_off, n_rows, max_rows) -> _KvSeqs:
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_seqs, max_pages]")
    n, width = page_table.shape
    index = cache.index
    return _KvSeqs(_ids("page_table", page_table, (n, width), index), _ids("kv_len", kv_len, (n,), index),
                   None if row_off is None else _ids("row_off", row_off, (n + 1,), index), n_rows, n, width, max_rows)


def _rows(name, x, heads, hd, index) -> int:
    """Row distance in elements of [n, heads, hd] rows whose heads lie side by side."""
    if x.dim() != 3 or x.shape[1] != heads or x.shape[2] != hd or x.get_device() != index:
        raise ValueError(f"{name} must be [rows, {heads}, {hd}] on the cache's device")
    if x.is_contiguous():
        return heads * hd
    st = x.stride()
    if st[2] != 1 or (st[1] != hd and heads != 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return st[0] if x.shape[0] > 1 else heads * hd


def kv_append(cache: KvCache, page_table, kv_len, k, v, row_off=None, max_rows: int = 1, stream=None):
    """Write the rows k, v [n_rows, n_kv_heads, head_dim] (bf16 or float32; rows
    may be any multiple of 16 bytes apart) as the newest tokens of their
    sequences."""
    q = _seqs(cache, page_table, kv_len, row_off, k.shape[0], max_rows)
    ldk = _rows("k", k, cache.n_kv_heads, cache.head_dim, cache.index)
    ldv = _rows("v", v, cache.n_kv_heads, cache.head_dim, cache.index)
    if v.shape[0] != k.shape[0] or v.dtype != k.dtype:
        raise ValueError("k and v must have the same rows and dtype")
    _check(_lib().mlora_kv_append(cache._ref, byref(q), _dtype(k.dtype), k.data_ptr(), ldk, v.data_ptr(), ldv,
                                  _on(cache.index, stream)))


def kv_read(cache: KvCache, page_table, kv_len, n_rows: int, row_off=None, max_rows: int = 1, dtype=None, stream=None):
    """(k, v) [n_rows, n_kv_heads, head_dim] of the newest tokens, as float32 (default) or bf16."""
    dtype = torch.float32 if dtype is None else dtype
    q = _seqs(cache, page_table, kv_len, row_off, n_rows, max_rows)
    shape = (n_rows, cache.n_kv_heads, cache.head_dim)
    ko = _empty(shape, dtype, cache.device, stream)
    vo = _empty(shape, dtype, cache.device, stream)
    _check(_lib().mlora_kv_read(cache._ref, byref(q), _dtype(dtype), ko.data_ptr(), vo.data_ptr(), _on(cache.index, stream)))
    return ko, vo


def kv_attention(cache: KvCache, page_table, kv_len, q, max_len: int, row_off=None, max_rows: int = 1, scale=None,
                 out=None, lse=None, workspace=None, stream=None):
    """Attention of the rows q [n_rows, n_heads, head_dim] over their sequences'
    cached positions up to their own.  Returns (out like q, lse float32
    [n_rows, n_heads]); scale defaults to 1 / sqrt(head_dim).  Without a
    workspace one is allocated for the call.  Nothing is recorded for autograd,
    whatever q, out or lse require."""
    if q.dim() != 3:
        raise ValueError("q must be [rows, heads, head_dim]")
    n_rows, heads, hd = q.shape
    s = _seqs(cache, page_table, kv_len, row_off, n_rows, max_rows)
    ldq = _rows("q", q, heads, cache.head_dim, cache.index)
    if out is None:
        out = _empty(q.shape, q.dtype, cache.device, stream)
    elif out.dtype != q.dtype or out.shape[0] != n_rows:
        raise ValueError("out must have q's rows and dtype")
    ldo = _rows("out", out, heads, cache.head_dim, cache.index)
    if lse is None:
        lse = _empty((n_rows, heads), torch.float32, cache.device, stream)
    elif lse.dtype is not _FLOAT32 or lse.shape != (n_rows, heads) or not lse.is_contiguous() or \
            lse.get_device() != cache.index:
        raise ValueError("lse must be a contiguous float32 [rows, heads] tensor on the cache's device")
    if workspace is None:
        workspace = _empty(WORKSPACE_BYTES, torch.uint8, cache.device, stream)
    elif not workspace.is_contiguous() or workspace.get_device() != cache.index:
        raise ValueError("workspace must be contiguous and on the cache's device")
    a = _KvAttn(q.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), ldq, ldo,
                workspace.numel() * workspace.element_size(), max_len, _dtype(q.dtype), heads,
                1.0 / math.sqrt(hd) if scale is None else scale)
    _check(_lib().mlora_kv_attention(cache._ref, byref(s), byref(a), _on(cache.index, stream)))
    return out, lse


def _context(h, caches, tokens, page_table, kv_len, max_len, row_off, max_rows, workspace, stream):
    if len(caches) != h.n_layers:
        raise ValueError(f"{h.n_layers} caches are needed, one per layer")
    c0 = caches[0]
    if workspace is None:
        workspace = _empty(WORKSPACE_BYTES, torch.uint8, c0.device, stream)
    elif not workspace.is_contiguous() or workspace.get_device() != c0.index:
        raise ValueError("workspace must be contiguous and on the caches' device")
    if any(c.index != c0.index for c in caches):
        raise ValueError("the caches must be on one device")
    arr = (_KvCache * len(caches))(*[c._c for c in caches])
    ctx = _TfContext(arr, _seqs(c0, page_table, kv_len, row_off, tokens.numel(), max_rows), workspace.data_ptr(),
                     workspace.numel() * workspace.element_size(), max_len)
    ctx._keep = (arr, workspace)
    return ctx


def tf_forward_cached(h, caches, tokens, targets, adapter_ids, page_table, kv_len, max_len: int, row_off=None,
                      max_rows: int = 1, workspace=None, logprobs_out=None, stream=None):
    """Forward of the sequences' newest rows over one cache per layer, which gets
    their keys and values; returns the targets' logprobs (targets None: only
    the caches are filled).  Without a workspace one is allocated for the call."""
    ctx = _context(h, caches, tokens, page_table, kv_len, max_len, row_off, max_rows, workspace, stream)
    c0 = caches[0]
    n = tokens.numel()
    if targets is not None and logprobs_out is None:
        logprobs_out = _empty(n, torch.float32, c0.device, stream)
    b = _TfBatch(n, _ids("tokens", tokens, (n,), c0.index),
                 None if targets is None else _ids("targets", targets, (n,), c0.index), None,
                 _ids("adapter_ids", adapter_ids, (n,), c0.index))
    _check(_lib().mlora_tf_forward_cached(h.ptr, byref(b), byref(ctx),
                                          None if targets is None else _out("logprobs_out", logprobs_out, n, c0.index),
                                          _on(c0.index, stream)))
    return logprobs_out if targets is not None else None


def tf_sample_cached(h, caches, tokens, adapter_ids, uniforms, page_table, kv_len, max_len: int, row_off=None,
                     max_rows: int = 1, workspace=None, next_out=None, logprob_out=None, stream=None):
    """The same, and the next token of every sequence from its last row:
    returns (next int32 [n_seqs], its logprob float32 [n_seqs])."""
    ctx = _context(h, caches, tokens, page_table, kv_len, max_len, row_off, max_rows, workspace, stream)
    c0 = caches[0]
    n, m = tokens.numel(), page_table.shape[0]
    if next_out is None:
        next_out = _empty(m, torch.int32, c0.device, stream)
    if logprob_out is None:
        logprob_out = _empty(m, torch.float32, c0.device, stream)
    b = _TfBatch(n, _ids("tokens", tokens, (n,), c0.index), None, None, _ids("adapter_ids", adapter_ids, (n,), c0.index))
    _check(_lib().mlora_tf_sample_cached(h.ptr, byref(b), byref(ctx), _out("uniforms", uniforms, m, c0.index),
                                         _ids("next_out", next_out, (m,), c0.index),
                                         _out("logprob_out", logprob_out, m, c0.index), _on(c0.index, stream)))
    return next_out, logprob_out


def kv_check_status(cache: KvCache, stream=None) -> int:
    """Synchronise, return and clear the cache's status: 0, -2 (E_RANGE), or -5
    (E_TIMEOUT: a bounded device wait gave up).  The word is read and cleared in
    the order of `stream` (None: the current one): a bit that later work there
    raises is kept.  Calls of the cache on other streams should have ended."""
    stream = stream or torch.cuda.current_stream(cache.index)
    with torch.cuda.stream(stream):
        bad = int(cache.status.item())
        if bad:
            cache.status.zero_()
    return -5 if bad & 2 else -2 if bad & 1 else 0
