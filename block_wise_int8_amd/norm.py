"""The root-mean-square norm that feeds the 8-bit layers (``include/blockint8_norm.h``)."""
from __future__ import annotations

import torch

import block_wise_int8_amd as _bi8

from . import _call as c

__all__ = ["rmsnorm_quant"]


def declare(lib) -> None:
    vp, i64, i32 = c.VP, c.I64, c.I32
    args = [vp, i64, vp, i64, vp, c.F64, i64, i64, i32, vp, i64, vp, vp, vp, vp]
    c.declare(lib, "blockint8_rmsnorm_quant", args)
    c.declare(lib, "blockint8_rmsnorm_quant_fp8", args)


def rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                  dtype: torch.dtype | None = None, xq: torch.Tensor | None = None, xs: torch.Tensor | None = None,
                  h: torch.Tensor | None = None, y: torch.Tensor | None = None, return_y: bool = False):
    """h = x + residual, its RMS norm times ``weight``, quantised per token and 128 columns.

    ``x`` and ``residual`` are bf16 [M, H] (rows may lie further apart),
    ``weight`` bf16 [H].  ``dtype`` (torch.int8, the default, or
    torch.float8_e4m3fn; the type of ``xq`` when that is given) is the type of
    the codes: what ``gemm`` or ``gemm_fp8`` reads.

    Returns ``(xq [M, H], xs float32 [M, ceil(H/128)])``, followed by ``h``
    bf16 [M, H] when there is a residual and by ``y``, the norm in bf16, when
    ``y`` is given or ``return_y`` set.  ``h`` may be ``x`` or ``residual``
    itself: the sum is then formed in place."""
    dev = c.device_of(x, "x")
    M, H, ldx = c.rows(x, "x", dev)
    c.dense(weight, "weight", dev, torch.bfloat16, (H,))
    if dtype is None:
        dtype = torch.int8 if xq is None else xq.dtype
    if dtype not in (torch.int8, torch.float8_e4m3fn):
        raise TypeError("the codes are torch.int8 or torch.float8_e4m3fn (got %s)" % dtype)
    ldr = ldh = H
    if residual is not None:
        shape = x.shape
        ldr = c.rows_like(residual, "residual", dev, shape)
        if h is None:
            h = torch.empty((M, H), dtype=torch.bfloat16, device=dev)
        else:
            ldh = c.rows_like(h, "h", dev, shape)
    elif h is not None:
        raise ValueError("h is the sum with a residual: there is none")
    xq = c.output(xq, "xq", dev, dtype, (M, H))
    xs = c.output(xs, "xs", dev, torch.float32, (M, -(-H // _bi8.BLOCK)))
    if y is not None or return_y:
        y = c.output(y, "y", dev, torch.bfloat16, (M, H))
    lib = _bi8.load()
    fn = lib.blockint8_rmsnorm_quant if dtype == torch.int8 else lib.blockint8_rmsnorm_quant_fp8
    _bi8._check(c.call(fn, dev, x.data_ptr(), ldx, c.ptr(residual), ldr, weight.data_ptr(), eps, M, H, 128, c.ptr(h),
                       ldh, c.ptr(y), xq.data_ptr(), xs.data_ptr()))
    out = (xq, xs)
    if residual is not None:
        out += (h,)
    if y is not None:
        out += (y,)
    return out
