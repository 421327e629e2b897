"""Argument checks and the call itself, shared by the binding's modules.

A decoding step calls these functions thousands of times a second on a few
tokens each, so the checks stay on cheap tensor queries: device indices
instead of device objects, and the current stream's handle without a stream
object around it.
"""
from __future__ import annotations

import ctypes

import torch

_Tensor = torch.Tensor


def device_of(t, name: str) -> int:
    """Index of the HIP device that a call's tensors have to share, from its first tensor."""
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a HIP device (got %s); there is no CPU path" % (name, t.device))
    return t.get_device()


def _elsewhere(t, name: str, dev: int):
    return ValueError("%s must be on cuda:%d (got %s)" % (name, dev, t.device))


def rows(t, name: str, dev: int, dtype: torch.dtype = torch.bfloat16):
    """Check a 2-D tensor whose rows are contiguous and may lie further apart: (rows, columns, leading dimension)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            shape = t.shape
            if len(shape) == 2:
                M, K = shape
                return M, K, K
    except AttributeError:
        pass
    if not isinstance(t, _Tensor) or t.dim() != 2 or t.dtype is not dtype:
        raise TypeError("%s must be a 2-D %s tensor" % (name, str(dtype).replace("torch.", "")))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    M, K = t.shape
    ld, step = t.stride()
    if step != 1 and K > 1:
        raise ValueError("%s rows must be contiguous (stride(1) == 1)" % name)
    if M <= 1:
        ld = K
    elif ld < K:
        raise ValueError("%s rows overlap (stride(0) = %d, %d columns)" % (name, ld, K))
    return M, K, ld


def rows_like(t, name: str, dev: int, shape) -> int:
    """``rows`` of a bf16 tensor of the given shape: its leading dimension."""
    try:
        if t.shape == shape and t.dtype is torch.bfloat16 and t.get_device() == dev and t.is_contiguous():
            return shape[1]
    except AttributeError:
        pass
    M, K, ld = rows(t, name, dev)
    if (M, K) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), (M, K)))
    return ld


def dense(t, name: str, dev: int, dtype: torch.dtype, shape: tuple):
    """Check a contiguous tensor of the given type and shape (None: any size on that axis)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t
    except AttributeError:
        pass
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    got = t.shape
    if got != shape and (len(got) != len(shape) or any(w is not None and w != n for n, w in zip(got, shape))):
        raise ValueError("%s must have shape %s (got %s)" % (name, shape, tuple(got)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def matrix(t, name: str, dev: int, dtype: torch.dtype, columns: int | None = None):
    """Check a contiguous 2-D tensor of the given type (and columns): its shape."""
    try:
        shape = t.shape
        if (t.dtype is dtype and len(shape) == 2 and (columns is None or shape[1] == columns)
                and t.get_device() == dev and t.is_contiguous()):
            return shape
    except AttributeError:
        pass
    return dense(t, name, dev, dtype, (None, columns)).shape


def output(t, name: str, dev: int, dtype: torch.dtype, shape: tuple):
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return dense(t, name, dev, dtype, shape)


def routing(route, x, logits, renormalize: bool, E: int, k: int):
    """A given routing of x's tokens, checked: (topk_weights, sorted_token, expert_offsets, row_of)."""
    if logits is not None or renormalize:
        raise ValueError("a given routing takes no logits and is not renormalised")
    dev, T = device_of(x, "x"), x.shape[0]
    _, weights, sorted_token, offsets, row_of = route
    return (dense(weights, "topk_weights", dev, torch.float32, (T, k)),
            dense(sorted_token, "sorted_token", dev, torch.int32, (T * k,)),
            dense(offsets, "expert_offsets", dev, torch.int32, (E + 1,)),
            dense(row_of, "row_of", dev, torch.int32, (T, k)))


def scratch(t, dev: int):
    """(pointer, bytes) of an optional workspace of any type."""
    if t is None:
        return None, 0
    if not isinstance(t, _Tensor) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on cuda:%d" % dev)
    return t.data_ptr(), t.nbytes


def ptr(t):
    return None if t is None else t.data_ptr()


_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def call(fn, dev: int, *args) -> int:
    """fn(*args, stream) on the tensors' device and its current stream: the status."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fn(*args, _raw_stream(dev))
    return fn(*args, _raw_stream(dev))


VP, I64, I32, F64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double


def declare(lib: ctypes.CDLL, name: str, argtypes: list, restype=ctypes.c_int32) -> None:
    f = getattr(lib, name)
    f.argtypes = argtypes
    f.restype = restype
