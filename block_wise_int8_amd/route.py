"""The router with scores, a bias and groups of experts (``include/blockint8_route.h``)."""
from __future__ import annotations

import torch

import block_wise_int8_amd as _bi8

from . import _call as c

__all__ = ["moe_route_grouped", "moe_route_grouped_workspace_size"]

_SCORES = {"softmax": 0, "sigmoid": 1}


def declare(lib) -> None:
    vp, i64, i32 = c.VP, c.I64, c.I32
    c.declare(lib, "blockint8_moe_route_grouped", [vp, i32, i64, vp, i64] + [i32] * 7 + [c.F64] + [vp] * 6 + [i64, vp])
    c.declare(lib, "blockint8_moe_route_grouped_workspace_size", [i64, i32], i64)
    c.declare(lib, "blockint8_moe_layer_fp8_routed", [i32, vp, i64] + [vp] * 9 + [i64] * 3 + [i32] * 4 + [vp, i64, vp])
    c.declare(lib, "blockint8_moe_layer_fp8_routed_workspace_size", [i64, i64, i64, i32, i32], i64)


def moe_route_grouped_workspace_size(T: int, E: int) -> int:
    """Bytes of workspace ``moe_route_grouped`` needs for up to T tokens (0: none)."""
    return int(_bi8.load().blockint8_moe_route_grouped_workspace_size(T, E))


def moe_route_grouped(logits: torch.Tensor, k: int, score: str = "softmax", bias: torch.Tensor | None = None,
                      groups: int = 1, topk_groups: int = 1, group_top: int = 1, renormalize: bool = False,
                      scale: float = 1.0, out=None, workspace: torch.Tensor | None = None):
    """The k best experts of each token, their weights and the dispatch order.

    ``logits`` is float32 or bfloat16 [T, E] (rows may lie further apart), E up
    to 1024, k up to 32.  ``score``: "softmax" or "sigmoid".  ``bias`` float32 [E]
    is added to the scores for the choice, not to the weights.  With ``groups`` >
    1 the experts are chosen from the ``topk_groups`` groups with the largest
    score (``group_top`` 1) or sum of two largest scores (2), bias included.
    Weights are divided by their sum with ``renormalize``, then multiplied by
    ``scale``.  Ties go to the lower index.

    Returns ``(topk_ids int32 [T, k], topk_weights float32 [T, k], sorted_token
    int32 [T*k], expert_offsets int32 [E+1], row_of int32 [T, k])`` as
    ``moe_route`` does, written into ``out`` (a tuple of those five tensors) when
    given: what ``moe_layer`` and ``moe_layer_fp8`` take as ``route``.
    ``workspace``: a contiguous tensor of any type on the device, of
    ``moe_route_grouped_workspace_size`` bytes or more (a fresh one when not
    given); calls that share one must not overlap in time."""
    dev = c.device_of(logits, "logits")
    bf16 = logits.dtype is torch.bfloat16
    T, E, ldl = c.rows(logits, "logits", dev, torch.bfloat16 if bf16 else torch.float32)
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid' (got %r)" % (score,))
    if bias is not None:
        c.dense(bias, "bias", dev, torch.float32, (E,))
    if out is None:
        out = (None,) * 5
    ids = c.output(out[0], "topk_ids", dev, torch.int32, (T, k))
    weights = c.output(out[1], "topk_weights", dev, torch.float32, (T, k))
    sorted_token = c.output(out[2], "sorted_token", dev, torch.int32, (T * k,))
    offsets = c.output(out[3], "expert_offsets", dev, torch.int32, (E + 1,))
    row_of = c.output(out[4], "row_of", dev, torch.int32, (T, k))
    lib = _bi8.load()
    if workspace is None:
        need = lib.blockint8_moe_route_grouped_workspace_size(T, E)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    wsp, nbytes = c.scratch(workspace, dev)
    _bi8._check(c.call(lib.blockint8_moe_route_grouped, dev, logits.data_ptr(), 1 if bf16 else 0, ldl, c.ptr(bias), T, E,
                       k, _SCORES[score], groups, topk_groups, group_top, 1 if renormalize else 0, scale, ids.data_ptr(),
                       weights.data_ptr(), sorted_token.data_ptr(), offsets.data_ptr(), row_of.data_ptr(), wsp, nbytes))
    return ids, weights, sorted_token, offsets, row_of
