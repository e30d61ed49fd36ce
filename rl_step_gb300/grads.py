"""Python binding of mlora_clip_grads and mlora_orthogonalize (include/mlora.h):
the gradient norm of each group of tensors, and clipping; updates made orthogonal.
Argument marshalling only.

    gs = GradSet(grads, groups)           # groups: an adapter id per tensor (None: one group)
    norms = clip_grads(gs, 1.0)           # in place; float32 [n_groups], device
    ms = MatrixSet(updates, out=outs)     # LoRA factors' gradients or momenta, 2-D
    orthogonalize(ms, steps=5)            # Newton-Schulz products
"""
from __future__ import annotations

import ctypes
from ctypes import POINTER, byref, c_float, c_int32, c_int64, c_void_p
from typing import Optional, Sequence

import torch

from . import _check, load_library
from .kv import _empty, _on

__all__ = ["GradSet", "clip_grads", "MatrixSet", "orthogonalize"]


class _GradSet(ctypes.Structure):
    _fields_ = [("grads", POINTER(c_void_p)), ("out", POINTER(c_void_p)), ("sizes", POINTER(c_int64)),
                ("groups", POINTER(c_int32)), ("n_tensors", c_int32), ("n_groups", c_int32), ("dtype", c_int32)]


class _MatrixSet(ctypes.Structure):
    _fields_ = [("src", POINTER(c_void_p)), ("dst", POINTER(c_void_p)), ("rows", POINTER(c_int64)),
                ("cols", POINTER(c_int64)), ("n_matrices", c_int32), ("dtype", c_int32)]


class _NewtonSchulz(ctypes.Structure):
    _fields_ = [("a", c_float), ("b", c_float), ("c", c_float), ("eps", c_float), ("steps", c_int32)]


_SIGNATURES = {
    "mlora_orthogonalize": (c_int32, [POINTER(_MatrixSet), POINTER(_NewtonSchulz), c_void_p]),
    "mlora_clip_grads_workspace": (c_int64, [POINTER(_GradSet)]),
    "mlora_clip_grads": (c_int32, [POINTER(_GradSet), c_float, c_void_p, c_void_p, c_int64, c_void_p]),
}

_grads_lib = None


def _lib():
    global _grads_lib
    if _grads_lib is None:
        lib = load_library()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _grads_lib = lib
    return _grads_lib


def _no_overlap(ptrs, outs, sizes, width):
    """What a call writes must overlap nothing else of its set (a tensor listed twice would be scaled twice)."""
    spans = [(o, o + n * width, True) for o, n in zip(outs, sizes) if n]
    spans += [(p, p + n * width, False) for p, o, n in zip(ptrs, outs, sizes) if n and p != o]
    spans.sort()
    written = seen = 0                            # ends so far
    for start, end, writes in spans:
        if start < (seen if writes else written):
            raise ValueError("an output overlaps another tensor of the set")
        if end > seen:
            seen = end
        if writes and end > written:
            written = end


class GradSet:
    """The tensors of repeated clip_grads calls: contiguous CUDA tensors of one
    dtype (float32 or bf16), an optional group of each, optional outputs (None:
    in place).  Keeps the tensors alive, and a workspace for the calls on the
    stream it was made on (other streams' and captured calls take one each).
    Making one takes 1 to 2 us of host time a tensor, many times a call's: keep it
    where the same tensors are clipped step after step."""

    def __init__(self, grads: Sequence, groups: Optional[Sequence[int]] = None, n_groups: Optional[int] = None,
                 out: Optional[Sequence] = None):
        self.grads, self.out = list(grads), None if out is None else list(out)
        n = len(self.grads)
        if n == 0:
            raise ValueError("no tensors")
        dtype, self.device = self.grads[0].dtype, self.grads[0].device
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"dtype {dtype}: bfloat16 or float32 is needed")
        if self.out is not None and [tuple(o.shape) for o in self.out] != [tuple(g.shape) for g in self.grads]:
            raise ValueError("out must have the tensors' shapes")
        for t in self.grads + (self.out or []):
            if t.dtype != dtype or t.device != self.device or not t.is_cuda or not t.is_contiguous():
                raise ValueError("tensors must be contiguous CUDA tensors of one dtype on one device")
        ptrs = [t.data_ptr() for t in self.grads]
        outs = None if self.out is None else [t.data_ptr() for t in self.out]
        sizes = [t.numel() for t in self.grads]
        _no_overlap(ptrs, outs or ptrs, sizes, self.grads[0].element_size())
        if groups is not None and len(groups) != n:
            raise ValueError("groups must name a group for each tensor")
        self.n_groups = n_groups if n_groups is not None else (1 if groups is None else max(groups) + 1)
        self._arrays = ((c_void_p * n)(*ptrs), None if outs is None else (c_void_p * n)(*outs), (c_int64 * n)(*sizes),
                        None if groups is None else (c_int32 * n)(*groups))
        self._c = _GradSet(self._arrays[0], self._arrays[1], self._arrays[2], self._arrays[3], n, self.n_groups,
                           0 if dtype == torch.bfloat16 else 1)
        self._ref = byref(self._c)
        self.index = self.grads[0].get_device()
        self._bytes = int(_lib().mlora_clip_grads_workspace(self._ref))
        if self._bytes == 0:                      # refused: raise its message
            _check(_lib().mlora_clip_grads(self._ref, 0.0, None, None, 0, None))
        with torch.cuda.device(self.index):
            self._stream = torch.cuda.current_stream().cuda_stream
            self._workspace = _empty(self._bytes, torch.uint8, self.device, None)


def _capturing(stream) -> bool:
    """Whether the stream of the call (None: the current one) is being captured."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def clip_grads(gs: GradSet, max_norm: float, norms_out=None, stream=None):
    """Clip each group of gs to max_norm; returns the norms before clipping
    (float32 [n_groups]).  Autograd sees nothing of it: tensors clipped in place
    keep their version counters."""
    handle = _on(gs.index, stream)
    if handle == gs._stream and not _capturing(stream):
        workspace = gs._workspace
    else:
        workspace = _empty(gs._bytes, torch.uint8, gs.device, stream)
    if norms_out is None:
        norms_out = _empty(gs.n_groups, torch.float32, gs.device, stream)
    elif norms_out.dtype is not torch.float32 or norms_out.numel() != gs.n_groups or \
            not norms_out.is_contiguous() or norms_out.get_device() != gs.index:
        raise ValueError("norms_out must be a contiguous float32 tensor with a value for each group")
    _check(_lib().mlora_clip_grads(gs._ref, max_norm, norms_out.data_ptr(), workspace.data_ptr(), gs._bytes,
                                   handle))
    return norms_out


class MatrixSet:
    """The matrices of repeated orthogonalize calls: contiguous 2-D CUDA tensors of
    one dtype (float32 or bf16) whose shorter side is at most 64, and optional outputs
    (None: in place).  Keeps the tensors alive.  Making one takes about 3 us of host
    time a matrix, more than many calls do: keep it where the same tensors are taken step
    after step.  (tf_read_adapter returns new tensors; copy them into a set's own.)"""

    def __init__(self, mats: Sequence, out: Optional[Sequence] = None):
        self.mats, self.out = list(mats), None if out is None else list(out)
        n = len(self.mats)
        if n == 0:
            raise ValueError("no matrices")
        dtype, self.device = self.mats[0].dtype, self.mats[0].device
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"dtype {dtype}: bfloat16 or float32 is needed")
        if any(m.dim() != 2 for m in self.mats):
            raise ValueError("matrices have two dimensions")
        if self.out is not None and [tuple(o.shape) for o in self.out] != [tuple(m.shape) for m in self.mats]:
            raise ValueError("out must have the matrices' shapes")
        for t in self.mats + (self.out or []):
            if t.dtype != dtype or t.device != self.device or not t.is_cuda or not t.is_contiguous():
                raise ValueError("matrices must be contiguous CUDA tensors of one dtype on one device")
        ptrs = [t.data_ptr() for t in self.mats]
        outs = None if self.out is None else [t.data_ptr() for t in self.out]
        _no_overlap(ptrs, outs or ptrs, [t.numel() for t in self.mats], self.mats[0].element_size())
        shapes = [t.shape for t in self.mats]
        self._arrays = ((c_void_p * n)(*ptrs), None if outs is None else (c_void_p * n)(*outs),
                        (c_int64 * n)(*[s[0] for s in shapes]), (c_int64 * n)(*[s[1] for s in shapes]))
        self._c = _MatrixSet(*self._arrays, n, 0 if dtype == torch.bfloat16 else 1)
        self._ref = byref(self._c)
        self.index = self.mats[0].get_device()


def orthogonalize(ms: MatrixSet, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  stream=None):
    """x <- m / (|m| + eps), then `steps` times x <- a x + (b A + c A A) x with A = x x^T
    over the shorter side, for each matrix; returns the outputs (the matrices
    themselves where the set has none).  Autograd sees nothing of it."""
    a, b, c = coefficients
    _check(_lib().mlora_orthogonalize(ms._ref, byref(_NewtonSchulz(a, b, c, eps, steps)), _on(ms.index, stream)))
    return ms.mats if ms.out is None else ms.out
