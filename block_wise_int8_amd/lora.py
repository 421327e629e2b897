"""Low-rank adapters of many requests beside a shared projection (``include/blockint8_lora.h``)."""
from __future__ import annotations

import ctypes

import torch

import block_wise_int8_amd as _bi8

from . import _call as c

__all__ = ["lora_add", "lora_add_workspace_size"]


def declare(lib) -> None:
    vp, i64, i32 = c.VP, c.I64, c.I32
    c.declare(lib, "blockint8_lora_add", [vp, i64, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, i32,
                                          ctypes.POINTER(i64), vp, i64, vp])
    c.declare(lib, "blockint8_lora_add_workspace_size", [i64, i64, i32, i32], i64)


def lora_add_workspace_size(M: int, K: int, R: int, parts: int = 1) -> int:
    """Bytes of workspace ``lora_add`` needs for up to M rows of K columns and adapters of rank R in each part."""
    return int(_bi8.load().blockint8_lora_add_workspace_size(M, K, R, parts))


def lora_add(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapter: torch.Tensor,
             scales: torch.Tensor | None = None, parts=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m] += scales[e] (x[m] a[e]^T) b[e]^T with e = adapter[m], in place; returns ``y``.

    ``y`` is bf16 [M, N], the output of a projection of ``x`` bf16 [M, K] (rows
    of either may lie further apart).  ``a`` is bf16 [L, R, K], ``b`` bf16 [L, N,
    R] with R a multiple of 8; ``scales`` float32 [L].  ``adapter`` is int32 [M]: a
    row whose value lies outside [0, L) is left as it was.  ``parts``: the widths
    of the projections side by side in ``y`` (query, key, value), of which each
    has R ranks of its own: ``a`` is [L, len(parts) * R, K] then, at most 256 ranks
    in all.  ``workspace``: a contiguous tensor of any type on the device, of
    ``lora_add_workspace_size`` bytes or more (a fresh one when not given); calls
    that share one must not overlap in time."""
    dev = c.device_of(y, "y")
    M, N, ldy = c.rows(y, "y", dev)
    rows, K, ldx = c.rows(x, "x", dev)
    if rows != M:
        raise ValueError("x must have %d rows (got %d)" % (M, rows))
    n = 1 if parts is None else len(parts)
    c.dense(b, "b", dev, torch.bfloat16, (None, N, None))
    L, _, R = b.shape
    c.dense(a, "a", dev, torch.bfloat16, (L, n * R, K))
    c.dense(adapter, "adapter", dev, torch.int32, (M,))
    if scales is not None:
        c.dense(scales, "scales", dev, torch.float32, (L,))
    lib = _bi8.load()
    if workspace is None:
        workspace = torch.empty(lib.blockint8_lora_add_workspace_size(M, K, R, n), dtype=torch.uint8, device=dev)
    wsp, nbytes = c.scratch(workspace, dev)
    _bi8._check(c.call(lib.blockint8_lora_add, dev, x.data_ptr(), ldx, a.data_ptr(), b.data_ptr(), c.ptr(scales),
                       adapter.data_ptr(), y.data_ptr(), ldy, M, N, K, L, R, n,
                       (ctypes.c_int64 * n)(*((N,) if parts is None else parts)), wsp, nbytes))
    return y
