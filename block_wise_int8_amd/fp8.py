"""The e4m3 form of the block-scaled linear and MoE layer (``include/blockint8_fp8.h``).

The functions of the int8 layer with ``torch.float8_e4m3fn`` codes in the place
of int8 ones: the same shapes, scales, blocks ([128, 128]) and errors.

Products are summed in binary32 but, in the tiled kernels, for the matrix core's
own sums of eight consecutive products, which it aligns to the largest and cuts
2^-13 below its leading bit (0.0003 of a product's output in norm, against the
0.0017 of its rounding to bf16).  The streaming kernel and the variant
GEMM_TILE_256X128_F16 hold every sum, the latter at half the matrix rate; the MoE
layer takes them for w13, whose result is quantised again, where the weights'
stream bounds it (its output is then 0.0017 from the 64-bit evaluation, else 0.0034).
"""
from __future__ import annotations

import torch

import block_wise_int8_amd as _bi8

from . import _call as c

__all__ = ["quant_act_fp8", "quant_act_gather_fp8", "silu_mul_quant_fp8", "quant_weight_fp8", "gemm_fp8",
           "gemm_fp8_workspace_size", "linear_fp8", "moe_gemm_fp8", "moe_gemm_silu_quant_fp8",
           "moe_gemm_fp8_workspace_size", "gemm_fp8_select", "moe_gemm_fp8_select", "moe_layer_fp8",
           "moe_layer_fp8_workspace_size", "moe_layer_fp8_select", "GEMM_TILE_128X128", "GEMM_TILE_256X128_F16"]

FP8 = torch.float8_e4m3fn
# kernel variants that the int8 GEMM does not have
GEMM_TILE_128X128 = 5
GEMM_TILE_256X128_F16 = 8   # the codes multiplied as f16 values


def declare(lib) -> None:
    vp, i64, i32 = c.VP, c.I64, c.I32
    c.declare(lib, "blockint8_quant_act_fp8", [vp, i64, i64, i64, i32, vp, vp, vp])
    c.declare(lib, "blockint8_quant_act_gather_fp8", [vp, i64, i64, vp, i64, i64, i32, vp, vp, vp])
    c.declare(lib, "blockint8_silu_mul_quant_fp8", [vp, i64, i64, i32, vp, vp, vp, vp])
    c.declare(lib, "blockint8_quant_weight_fp8", [vp, i64, i64, i64, i32, i32, vp, vp, vp])
    c.declare(lib, "blockint8_gemm_fp8", [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, i64, vp])
    c.declare(lib, "blockint8_gemm_fp8_workspace_size", [i64, i64, i64], i64)
    c.declare(lib, "blockint8_linear_fp8", [vp, i64, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, vp, vp, i64, vp])
    c.declare(lib, "blockint8_moe_gemm_fp8", [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, i32, vp, i64, vp])
    c.declare(lib, "blockint8_moe_gemm_silu_quant_fp8", [vp] * 7 + [i64, i64, i64, i32, i32, i32, vp])
    c.declare(lib, "blockint8_moe_layer_fp8", [vp, i64, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, i32, i32, i32, vp,
                                               i64, vp])
    c.declare(lib, "blockint8_moe_layer_fp8_variant", [i32] + lib.blockint8_moe_layer_fp8.argtypes)
    c.declare(lib, "blockint8_moe_layer_fp8_select", [i64, i64, i64, i32, i32])
    c.declare(lib, "blockint8_moe_layer_fp8_workspace_size", [i64, i64, i64, i32, i32], i64)
    c.declare(lib, "blockint8_gemm_fp8_variant", [i32] + lib.blockint8_gemm_fp8.argtypes)
    c.declare(lib, "blockint8_moe_gemm_fp8_variant", [i32] + lib.blockint8_moe_gemm_fp8.argtypes)
    c.declare(lib, "blockint8_gemm_fp8_select", [i64, i64, i64])
    c.declare(lib, "blockint8_moe_gemm_fp8_select", [i64, i64, i64, i32])
    c.declare(lib, "blockint8_moe_gemm_fp8_workspace_size", [i64, i64, i64, i32], i64)


def _blocks(n: int) -> int:
    return -(-n // _bi8.BLOCK)


def quant_act_fp8(x: torch.Tensor, xq: torch.Tensor | None = None, xs: torch.Tensor | None = None):
    """Dynamic quantisation of bf16 ``x`` [M, K], one scale per token and 128 columns.

    Returns ``(xq float8_e4m3fn [M, K], xs float32 [M, ceil(K/128)])``.  ``x``
    may have a row stride larger than K.
    """
    dev = c.device_of(x, "x")
    M, K, ldx = c.rows(x, "x", dev)
    xq = c.output(xq, "xq", dev, FP8, (M, K))
    xs = c.output(xs, "xs", dev, torch.float32, (M, _blocks(K)))
    _bi8._check(c.call(_bi8.load().blockint8_quant_act_fp8, dev, x.data_ptr(), M, K, ldx, 128, xq.data_ptr(),
                       xs.data_ptr()))
    return xq, xs


def quant_act_gather_fp8(x: torch.Tensor, rows: torch.Tensor, xq: torch.Tensor | None = None,
                         xs: torch.Tensor | None = None):
    """quant_act_fp8 of the rows ``x[rows]`` (bf16 [T, K], int32 indices [R])."""
    dev = c.device_of(x, "x")
    T, K, ldx = c.rows(x, "x", dev)
    c.dense(rows, "rows", dev, torch.int32, (None,))
    R = rows.shape[0]
    xq = c.output(xq, "xq", dev, FP8, (R, K))
    xs = c.output(xs, "xs", dev, torch.float32, (R, _blocks(K)))
    _bi8._check(c.call(_bi8.load().blockint8_quant_act_gather_fp8, dev, x.data_ptr(), T, ldx, rows.data_ptr(), R, K,
                       128, xq.data_ptr(), xs.data_ptr()))
    return xq, xs


def silu_mul_quant_fp8(h: torch.Tensor, aq: torch.Tensor | None = None, as_: torch.Tensor | None = None,
                       return_a: bool = False):
    """h = [gate | up] bf16 [R, 2I] -> (aq float8_e4m3fn [R, I], as float32 [R, ceil(I/128)][, a bf16 [R, I]])."""
    dev = c.device_of(h, "h")
    R, two_i = c.matrix(h, "h", dev, torch.bfloat16)
    if two_i % 2:
        raise ValueError("h must have an even number of columns (gate | up)")
    I = two_i // 2
    aq = c.output(aq, "aq", dev, FP8, (R, I))
    as_ = c.output(as_, "as_", dev, torch.float32, (R, _blocks(I)))
    a = torch.empty((R, I), dtype=torch.bfloat16, device=dev) if return_a else None
    _bi8._check(c.call(_bi8.load().blockint8_silu_mul_quant_fp8, dev, h.data_ptr(), R, I, 128, aq.data_ptr(),
                       as_.data_ptr(), c.ptr(a)))
    return (aq, as_, a) if return_a else (aq, as_)


def quant_weight_fp8(w: torch.Tensor):
    """Block quantisation of a bf16 weight [N, K] -> (float8_e4m3fn [N, K], float32 [ceil(N/128), ceil(K/128)])."""
    dev = c.device_of(w, "w")
    N, K, ldw = c.rows(w, "w", dev)
    wq = torch.empty((N, K), dtype=FP8, device=dev)
    ws = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=dev)
    _bi8._check(c.call(_bi8.load().blockint8_quant_weight_fp8, dev, w.data_ptr(), N, K, ldw, 128, 128, wq.data_ptr(),
                       ws.data_ptr()))
    return wq, ws


def gemm_fp8_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace ``gemm_fp8`` uses for an M x N x K problem (0: none)."""
    return int(_bi8.load().blockint8_gemm_fp8_workspace_size(M, N, K))


def gemm_fp8(xq: torch.Tensor, xs: torch.Tensor, w: torch.Tensor, ws: torch.Tensor,
             bias: torch.Tensor | None = None, y: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, variant: int | None = None) -> torch.Tensor:
    """Block-scaled e4m3 GEMM ``y = x . W^T (+ bias)`` -> bf16 [M, N].

    ``workspace`` (any contiguous tensor on the device, of at least
    ``gemm_fp8_workspace_size`` bytes) lets problems with few tiles split K
    between workgroups; calls that share one must not overlap in time.
    ``variant`` (one of ``GEMM_*``) runs a named kernel instead of the
    shape-based choice."""
    dev = c.device_of(xq, "xq")
    M, K = c.matrix(xq, "xq", dev, FP8)
    N, _ = c.matrix(w, "w", dev, FP8, K)
    c.dense(xs, "xs", dev, torch.float32, (M, _blocks(K)))
    c.dense(ws, "ws", dev, torch.float32, (_blocks(N), _blocks(K)))
    if bias is not None:
        c.dense(bias, "bias", dev, torch.bfloat16, (N,))
    y = c.output(y, "y", dev, torch.bfloat16, (M, N))
    wsp, nbytes = c.scratch(workspace, dev)
    _bi8._check(c.call(_bi8.load().blockint8_gemm_fp8_variant, dev, variant or 0, xq.data_ptr(), xs.data_ptr(),
                       w.data_ptr(), ws.data_ptr(), c.ptr(bias), y.data_ptr(), M, N, K, 128, 128, wsp, nbytes))
    return y


def linear_fp8(x: torch.Tensor, w: torch.Tensor, ws: torch.Tensor, bias: torch.Tensor | None = None,
               y: torch.Tensor | None = None, xq: torch.Tensor | None = None, xs: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The e4m3 linear with dynamic activation scales -> bf16 [M, N]: quant_act_fp8
    of bf16 ``x`` [M, K] into ``xq`` / ``xs`` (fresh tensors when not given;
    they hold the quantised activations on return), then gemm_fp8, through one
    C call.  ``workspace`` as for gemm_fp8."""
    dev = c.device_of(x, "x")
    M, K, ldx = c.rows(x, "x", dev)
    N, _ = c.matrix(w, "w", dev, FP8, K)
    KB = _blocks(K)
    c.dense(ws, "ws", dev, torch.float32, (_blocks(N), KB))
    if bias is not None:
        c.dense(bias, "bias", dev, torch.bfloat16, (N,))
    y = c.output(y, "y", dev, torch.bfloat16, (M, N))
    xq = c.output(xq, "xq", dev, FP8, (M, K))
    xs = c.output(xs, "xs", dev, torch.float32, (M, KB))
    wsp, nbytes = c.scratch(workspace, dev)
    _bi8._check(c.call(_bi8.load().blockint8_linear_fp8, dev, x.data_ptr(), ldx, w.data_ptr(), ws.data_ptr(),
                       c.ptr(bias), y.data_ptr(), M, N, K, 128, 128, xq.data_ptr(), xs.data_ptr(), wsp, nbytes))
    return y


def gemm_fp8_select(M: int, N: int, K: int) -> int:
    """The kernel variant (``GEMM_*``) that ``gemm_fp8`` runs for this shape without a workspace."""
    return int(_bi8.load().blockint8_gemm_fp8_select(M, N, K))


def moe_gemm_fp8_select(R: int, N: int, K: int, E: int) -> int:
    """The kernel variant (``GEMM_*``) that ``moe_gemm_fp8`` runs for this shape without a workspace."""
    return int(_bi8.load().blockint8_moe_gemm_fp8_select(R, N, K, E))


def moe_gemm_fp8_workspace_size(R: int, N: int, K: int, E: int) -> int:
    """Bytes of workspace ``moe_gemm_fp8`` can use for the grouped problem (0: none)."""
    return int(_bi8.load().blockint8_moe_gemm_fp8_workspace_size(R, N, K, E))


def moe_gemm_fp8(xq: torch.Tensor, xs: torch.Tensor, expert_offsets: torch.Tensor, w: torch.Tensor,
                 ws: torch.Tensor, y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 variant: int | None = None) -> torch.Tensor:
    """Grouped block-scaled e4m3 GEMM over expert-sorted rows -> bf16 [R, N].

    ``expert_offsets`` is int32 [E+1] on the device (rows [off[e], off[e+1])
    use expert e); ``w`` is float8_e4m3fn [E, N, K], ``ws`` float32 [E,
    ceil(N/128), ceil(K/128)].  ``workspace`` and ``variant`` as for gemm_fp8,
    with ``moe_gemm_fp8_workspace_size`` bytes."""
    dev = c.device_of(xq, "xq")
    R, K = c.matrix(xq, "xq", dev, FP8)
    c.dense(w, "w", dev, FP8, (None, None, K))
    E, N, _ = w.shape
    c.dense(expert_offsets, "expert_offsets", dev, torch.int32, (E + 1,))
    c.dense(xs, "xs", dev, torch.float32, (R, _blocks(K)))
    c.dense(ws, "ws", dev, torch.float32, (E, _blocks(N), _blocks(K)))
    y = c.output(y, "y", dev, torch.bfloat16, (R, N))
    wsp, nbytes = c.scratch(workspace, dev)
    _bi8._check(c.call(_bi8.load().blockint8_moe_gemm_fp8_variant, dev, variant or 0, xq.data_ptr(), xs.data_ptr(),
                       expert_offsets.data_ptr(), w.data_ptr(), ws.data_ptr(), y.data_ptr(), R, N, K, E, 128, 128, wsp,
                       nbytes))
    return y


def moe_gemm_silu_quant_fp8(xq: torch.Tensor, xs: torch.Tensor, expert_offsets: torch.Tensor, w13: torch.Tensor,
                            ws13: torch.Tensor, aq: torch.Tensor | None = None, as_: torch.Tensor | None = None):
    """The w13 grouped GEMM with the SiLU gating and requantisation as its
    epilogue: (aq float8_e4m3fn [R, I], as float32 [R, I/128]), what
    silu_mul_quant_fp8(moe_gemm_fp8(xq, xs, expert_offsets, w13, ws13)) gives
    up to the order of the products' sums.  w13 is float8_e4m3fn [E, 2I, K]
    (gate rows, then up rows); I % 128 == 0."""
    dev = c.device_of(xq, "xq")
    R, K = c.matrix(xq, "xq", dev, FP8)
    c.dense(w13, "w13", dev, FP8, (None, None, K))
    E, N, _ = w13.shape
    if N % 2:
        raise ValueError("w13 must have an even number of rows (gate, then up)")
    I = N // 2
    c.dense(expert_offsets, "expert_offsets", dev, torch.int32, (E + 1,))
    c.dense(xs, "xs", dev, torch.float32, (R, _blocks(K)))
    c.dense(ws13, "ws13", dev, torch.float32, (E, _blocks(N), _blocks(K)))
    aq = c.output(aq, "aq", dev, FP8, (R, I))
    as_ = c.output(as_, "as_", dev, torch.float32, (R, _blocks(I)))
    _bi8._check(c.call(_bi8.load().blockint8_moe_gemm_silu_quant_fp8, dev, xq.data_ptr(), xs.data_ptr(),
                       expert_offsets.data_ptr(), w13.data_ptr(), ws13.data_ptr(), aq.data_ptr(), as_.data_ptr(), R, I,
                       K, E, 128, 128))
    return aq, as_


def moe_layer_fp8_workspace_size(T: int, H: int, I: int, E: int, k: int) -> int:
    """Bytes of workspace ``moe_layer_fp8`` needs for T tokens."""
    return int(_bi8.load().blockint8_moe_layer_fp8_workspace_size(T, H, I, E, k))


def moe_layer_fp8_select(T: int, H: int, I: int, E: int, k: int) -> int:
    """The kernel variant (``GEMM_*``) that ``moe_layer_fp8`` runs for the w13 GEMM (0 for sizes it rejects)."""
    return int(_bi8.load().blockint8_moe_layer_fp8_select(T, H, I, E, k))


def moe_layer_fp8(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor, ws13: torch.Tensor, w2: torch.Tensor,
                  ws2: torch.Tensor, k: int, renormalize: bool = False, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, variant: int | None = None) -> torch.Tensor:
    """The e4m3 FusedMoE layer on the GPU, through one C call: route, gather +
    quantise, w13 grouped GEMM (moe_layer_fp8_select), SiLU gating + quantise,
    w2 grouped GEMM, weighted combine.  Where the w13 GEMM runs 256-row weight
    tiles and I % 128 == 0, it and the gating are one launch
    (moe_gemm_silu_quant_fp8).
    x bf16 [T, H]; logits fp32 [T, E]; w13 float8_e4m3fn [E, 2I, H]; w2
    float8_e4m3fn [E, H, I]; H and I multiples of 16.  ``workspace``: a
    contiguous, 256-byte aligned tensor of any type on the device, of
    ``moe_layer_fp8_workspace_size`` bytes or more (a fresh one when not
    given); calls that share one must not overlap in time.  ``variant``
    GEMM_TILE_256X128_F16 holds the w13 GEMM's sums, which the second quantiser
    reads, whatever its size.  Returns bf16 [T, H]."""
    dev = c.device_of(x, "x")
    T, H, ldx = c.rows(x, "x", dev)
    rows, E = c.matrix(logits, "logits", dev, torch.float32)
    if rows != T:
        raise ValueError("logits must have %d rows (got %d)" % (T, rows))
    c.dense(w13, "w13", dev, FP8, (E, None, H))
    N = w13.shape[1]
    if N % 2:
        raise ValueError("w13 must have an even number of rows (gate, then up)")
    I = N // 2
    c.dense(ws13, "ws13", dev, torch.float32, (E, _blocks(N), _blocks(H)))
    c.dense(w2, "w2", dev, FP8, (E, H, I))
    c.dense(ws2, "ws2", dev, torch.float32, (E, _blocks(H), _blocks(I)))
    out = c.output(out, "out", dev, torch.bfloat16, (T, H))
    lib = _bi8.load()
    if workspace is None:
        workspace = torch.empty(lib.blockint8_moe_layer_fp8_workspace_size(T, H, I, E, k), dtype=torch.uint8,
                                device=dev)
    wsp, nbytes = c.scratch(workspace, dev)
    _bi8._check(c.call(lib.blockint8_moe_layer_fp8_variant, dev, variant or 0, x.data_ptr(), ldx, logits.data_ptr(),
                       w13.data_ptr(), ws13.data_ptr(), w2.data_ptr(), ws2.data_ptr(), out.data_ptr(), T, H, I, E, k,
                       1 if renormalize else 0, 128, 128, wsp, nbytes))
    return out
