"""The norm and the rotation of query and key heads (``include/blockint8_heads.h``)."""
from __future__ import annotations

import ctypes

import torch

import block_wise_int8_amd as _bi8

from . import _call as c

__all__ = ["qk_norm_rope"]


def declare(lib) -> None:
    vp, i64, i32 = c.VP, c.I64, c.I32
    c.declare(lib, "blockint8_qk_norm_rope", [vp, i64, i64, i32, vp, i64, i64, i32, vp, vp, c.F64, vp, i64, vp, i64, i32,
                                              ctypes.POINTER(i32), i32, i64, i32, i32, vp, i64, i64, vp, i64, i64, vp])


def _heads(t, name: str, dev: int, T=None, H=None, D=None):
    """Check bf16 [tokens, heads, values] with contiguous values: its shape and strides."""
    try:
        if t.dtype is torch.bfloat16 and t.get_device() == dev:
            n, h, d = t.shape
            token, head, step = t.stride()
            if step == 1 and (T is None or (n == T and d == D and (H is None or h == H))):
                return n, h, d, token, head
    except (AttributeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 3:
        raise TypeError("%s must be a bfloat16 tensor [tokens, heads, values]" % name)
    if t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d (got %s)" % (name, dev, t.device))
    n, h, d = shape = t.shape
    if any(want is not None and want != got for want, got in zip((T, H, D), shape)):
        raise ValueError("%s must have shape %s (got %s)" % (name, (T, H, D), tuple(shape)))
    token, head, step = t.stride()
    if step != 1 and d > 1:
        raise ValueError("%s must have contiguous heads (stride(2) == 1)" % name)
    return n, h, d, token, head


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, table: torch.Tensor,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 sections=None, interleaved: bool = False, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None):
    """RMS norm of each head of ``q`` and ``k`` (where it has a weight) and its rotation by position.

    ``q`` is bf16 [T, Hq, D], ``k`` bf16 [T, Hk, D] or None, with any strides
    between tokens and heads: views of a projection's output.  ``q_weight`` and
    ``k_weight`` are bf16 [D].  ``table`` is float32 [P, rot]: the cosines, then
    the sines, of the rot/2 pairs at each position.  ``positions`` is int32 [T],
    or [axes, T] with ``sections``, how many pairs each axis turns.  Pairs are
    values i and i + rot/2, or 2i and 2i + 1 with ``interleaved``; values past
    rot are not turned.

    Returns ``(q_out, k_out)`` (``k_out`` None without ``k``): fresh dense tensors,
    or the given ones, which may be ``q`` and ``k`` themselves.  A token with a
    position outside [0, P) is left out: its outputs are not written."""
    dev = c.device_of(q, "q")
    T, Hq, D, q_token, q_head = _heads(q, "q", dev)
    Hk = k_token = k_head = k_out_token = k_out_head = 0
    if k is not None:
        _, Hk, _, k_token, k_head = _heads(k, "k", dev, T, None, D)
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight belong to k: there is none")
    P, rot = c.matrix(table, "table", dev, torch.float32)
    if q_weight is not None:
        c.dense(q_weight, "q_weight", dev, torch.bfloat16, (D,))
    if k_weight is not None:
        c.dense(k_weight, "k_weight", dev, torch.bfloat16, (D,))
    if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32 or positions.dim() not in (1, 2):
        raise TypeError("positions must be an int32 tensor [T] or [axes, T]")
    if positions.get_device() != dev:
        raise ValueError("positions must be on cuda:%d (got %s)" % (dev, positions.device))
    axes = positions.shape[0] if positions.dim() == 2 else 1
    if positions.shape[-1] != T or (T > 1 and positions.stride(-1) != 1):
        raise ValueError("positions must hold %d contiguous tokens an axis" % T)
    if sections is None:
        if axes != 1:
            raise ValueError("positions of %d axes need sections" % axes)
        sections = (rot // 2,)
    elif len(sections) != axes:
        raise ValueError("%d sections for positions of %d axes" % (len(sections), axes))
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    *_, q_out_token, q_out_head = _heads(q_out, "q_out", dev, T, Hq, D)
    if k is not None:
        if k_out is None:
            k_out = torch.empty((T, Hk, D), dtype=torch.bfloat16, device=dev)
        *_, k_out_token, k_out_head = _heads(k_out, "k_out", dev, T, Hk, D)
    _bi8._check(c.call(_bi8.load().blockint8_qk_norm_rope, dev, q.data_ptr(), q_token, q_head, Hq, c.ptr(k), k_token,
                       k_head, Hk, c.ptr(q_weight), c.ptr(k_weight), eps, table.data_ptr(), P, positions.data_ptr(),
                       positions.stride(0) if axes > 1 else 0, axes, (ctypes.c_int32 * axes)(*sections),
                       1 if interleaved else 0, T, D, rot, q_out.data_ptr(), q_out_token, q_out_head, c.ptr(k_out),
                       k_out_token, k_out_head))
    return q_out, k_out
