"""Python binding of include/mlora_logits.h: log-probabilities of given tokens
with entropy and the largest alternatives, and their gradient in the logits.
Argument marshalling only.

    r = token_logprobs(logits, targets, top=20)            # r.logprobs, .entropy, .lse, .top_ids, .top_logprobs
    d = token_logprobs_backward(logits, r.lse, r.entropy, targets, d_logprobs, d_entropy=..., ...)
    r = tf_forward_stats(h, tokens, targets, positions, adapter_ids, top=20)   # the transformer model's rows

Nothing is recorded for autograd: the gradient is a call of its own, as the
models' losses are.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple
from ctypes import POINTER, byref, c_float, c_int32, c_int64, c_void_p

import torch

from . import _check, load_library
from .kv import _dtype, _empty, _ids, _on, _stream_memory
from .transformer import _TfBatch

__all__ = ["TokenStats", "token_logprobs", "token_logprobs_backward", "tf_forward_stats"]

TokenStats = namedtuple("TokenStats", ["logprobs", "entropy", "lse", "top_ids", "top_logprobs"])


class _Logits(ctypes.Structure):
    _fields_ = [("logits", c_void_p), ("targets", c_void_p), ("status", c_void_p), ("stride", c_int64),
                ("n_rows", c_int64), ("vocab", c_int32), ("dtype", c_int32), ("scale", c_float), ("top", c_int32)]


class _TokenStats(ctypes.Structure):
    _fields_ = [("logprobs", c_void_p), ("entropy", c_void_p), ("lse", c_void_p), ("top_ids", c_void_p),
                ("top_logprobs", c_void_p)]


class _TokenGrads(ctypes.Structure):
    _fields_ = [("lse", c_void_p), ("entropy", c_void_p), ("top_ids", c_void_p), ("d_logprobs", c_void_p),
                ("d_entropy", c_void_p), ("d_lse", c_void_p), ("d_top", c_void_p)]


_SIGNATURES = {
    "mlora_token_logprobs": (c_int32, [POINTER(_Logits), POINTER(_TokenStats), c_void_p]),
    "mlora_token_logprobs_backward": (c_int32, [POINTER(_Logits), POINTER(_TokenGrads), c_void_p, c_int64, c_void_p]),
    "mlora_tf_forward_stats": (c_int32, [c_void_p, POINTER(_TfBatch), c_float, c_int32, POINTER(_TokenStats),
                                         c_void_p]),
}

_logits_lib = None


def _lib():
    global _logits_lib
    if _logits_lib is None:
        lib = load_library()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _logits_lib = lib
    return _logits_lib


def _row_stride(name, x):
    """Elements between the rows of x [n, vocab], whose own elements lie side by side."""
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [rows, vocab]")
    n, v = x.shape
    if v > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return x.stride(0) if n > 1 else v


def _values(name, t, shape, index):
    """Pointer of a float32 tensor of that shape, or None."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous float32 tensor {list(shape)} on the logits' device")
    return t.data_ptr()


def _rows(x, targets, scale, top, status):
    stride = _row_stride("logits", x)
    n, v = x.shape
    index = x.get_device()
    return _Logits(x.data_ptr(), None if targets is None else _ids("targets", targets, (n,), index),
                   None if status is None else _ids("status", status, (1,), index), stride, n, v, _dtype(x.dtype),
                   scale, top)


def token_logprobs(logits, targets=None, top: int = 0, scale: float = 1.0, status=None, stream=None) -> TokenStats:
    """Log-probabilities of int32 targets [n] in the rows of logits [n, vocab] (bf16
    or float32, rows any distance apart), and each row's entropy, log-sum-exp and
    `top` largest alternatives.  All float32 [n]; top_ids int32 and top_logprobs
    [n, top] (None where top is 0, logprobs None without targets).  scale: one
    over the temperature.  status: an int32 [1] whose bit 0 is raised by a target
    outside -1 .. vocab-1 (-1: a row without a target, NaN)."""
    c = _rows(logits, targets, scale, top, status)
    n, dev = logits.shape[0], logits.device
    handle = _on(logits.get_device(), stream)
    with _stream_memory(stream):
        lp = None if targets is None else torch.empty(n, dtype=torch.float32, device=dev)
        entropy = torch.empty(n, dtype=torch.float32, device=dev)
        lse = torch.empty(n, dtype=torch.float32, device=dev)
        ids = tops = None
        if top > 0:
            ids = torch.empty((n, top), dtype=torch.int32, device=dev)
            tops = torch.empty((n, top), dtype=torch.float32, device=dev)
    out = _TokenStats(None if lp is None else lp.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
                      None if ids is None else ids.data_ptr(), None if tops is None else tops.data_ptr())
    _check(_lib().mlora_token_logprobs(byref(c), byref(out), handle))
    return TokenStats(lp, entropy, lse, ids, tops)


def token_logprobs_backward(logits, lse, entropy=None, targets=None, d_logprobs=None, d_entropy=None, d_lse=None,
                            top_ids=None, d_top=None, scale: float = 1.0, out=None, status=None, stream=None):
    """The gradient in logits of a loss whose gradients in token_logprobs' results
    are d_logprobs, d_entropy, d_lse [n] and d_top [n, top] (None: none).  lse and
    entropy are the forward's, top_ids int32 [n, top] its alternatives or any ids
    (-1: none).  out: like logits, may be logits itself (None: a new contiguous
    tensor).  Rows of out that do not lie like the logits' (addresses equal modulo 32
    bytes) take several times as long: for logits that are a part of wider rows give an
    out that is one too."""
    top = 0
    if d_top is not None:
        if top_ids is None or d_top.dim() != 2:
            raise ValueError("d_top [n, top] needs the ids that it belongs to")
        top = d_top.shape[1]
    c = _rows(logits, targets, scale, top, status)
    n, index = logits.shape[0], logits.get_device()
    handle = _on(index, stream)
    if out is None:
        out = _empty(logits.shape, logits.dtype, logits.device, stream)
    elif out.dtype != logits.dtype or out.shape != logits.shape or out.get_device() != index:
        raise ValueError("out must have the logits' shape, dtype and device")
    g = _TokenGrads(_values("lse", lse, (n,), index), _values("entropy", entropy, (n,), index),
                    None if d_top is None else _ids("top_ids", top_ids, (n, top), index),
                    _values("d_logprobs", d_logprobs, (n,), index), _values("d_entropy", d_entropy, (n,), index),
                    _values("d_lse", d_lse, (n,), index), _values("d_top", d_top, (n, top), index))
    _check(_lib().mlora_token_logprobs_backward(byref(c), byref(g), out.data_ptr(), _row_stride("out", out), handle))
    return out


def tf_forward_stats(h, tokens, targets, positions, adapter_ids, top: int = 0, scale: float = 1.0,
                     stream=None) -> TokenStats:
    """token_logprobs' results for the rows of a batch of the transformer model
    (targets None: no logprobs)."""
    n, index, dev = tokens.numel(), tokens.get_device(), tokens.device
    handle = _on(index, stream)
    ids = lambda name, t: _ids(name, t, (n,), index)  # noqa: E731
    b = _TfBatch(n, ids("tokens", tokens), None if targets is None else ids("targets", targets),
                 ids("positions", positions), ids("adapter_ids", adapter_ids))
    new = lambda shape, dt=torch.float32: _empty(shape, dt, dev, stream)  # noqa: E731
    r = TokenStats(None if targets is None else new((n,)), new((n,)), new((n,)),
                   new((n, top), torch.int32) if top > 0 else None, new((n, top)) if top > 0 else None)
    out = _TokenStats(*[None if t is None else t.data_ptr() for t in r])
    _check(_lib().mlora_tf_forward_stats(h.ptr, byref(b), scale, top, byref(out), handle))
    return r
