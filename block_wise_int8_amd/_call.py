"""Argument checks and the call itself, shared by the binding's modules."""
from __future__ import annotations

import ctypes

import torch


def device_of(t: torch.Tensor, name: str) -> torch.device:
    """The HIP device that a call's tensors have to share, from its first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a HIP device (got %s); there is no CPU path" % (name, t.device))
    return t.device


def rows(t: torch.Tensor, name: str, dev: torch.device, dtype: torch.dtype = torch.bfloat16):
    """Check a 2-D tensor whose rows are contiguous and may lie further apart: (rows, columns, leading dimension)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype != dtype:
        raise TypeError("%s must be a 2-D %s tensor" % (name, str(dtype).replace("torch.", "")))
    if t.device != dev:
        raise ValueError("%s must be on %s (got %s)" % (name, dev, t.device))
    M, K = t.shape
    if K > 1 and t.stride(1) != 1:
        raise ValueError("%s rows must be contiguous (stride(1) == 1)" % name)
    ld = t.stride(0) if M > 1 else K
    if ld < K:
        raise ValueError("%s rows overlap (stride(0) = %d, %d columns)" % (name, ld, K))
    return M, K, ld


def dense(t: torch.Tensor, name: str, dev: torch.device, dtype: torch.dtype, shape: tuple) -> torch.Tensor:
    """Check a contiguous tensor of the given type and shape (None: any size on that axis)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.device != dev:
        raise ValueError("%s must be on %s (got %s)" % (name, dev, t.device))
    got = tuple(t.shape)
    if got != shape and (len(got) != len(shape) or any(w is not None and w != n for n, w in zip(got, shape))):
        raise ValueError("%s must have shape %s (got %s)" % (name, shape, got))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def output(t, name: str, dev: torch.device, dtype: torch.dtype, shape: tuple) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return dense(t, name, dev, dtype, shape)


def scratch(t, dev: torch.device):
    """(pointer, bytes) of an optional workspace of any type."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.device != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    return t.data_ptr(), t.numel() * t.element_size()


def ptr(t):
    return None if t is None else t.data_ptr()


def call(fn, dev: torch.device, *args) -> int:
    """fn(*args, stream) on the tensors' device and its current stream: the status."""
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    return fn(*args, torch.cuda.current_stream(dev).cuda_stream)


VP, I64, I32, F64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double


def declare(lib: ctypes.CDLL, name: str, argtypes: list, restype=ctypes.c_int32) -> None:
    f = getattr(lib, name)
    f.argtypes = argtypes
    f.restype = restype
