"""Oracle of the operators beside the 8-bit products -- test infrastructure.

Plain numpy in binary64, written from the definitions.  Shares no code with
``block_wise_int8_amd``.
"""
from __future__ import annotations

import numpy as np


def bf16(bits: np.ndarray) -> np.ndarray:
    """Values of bf16 bit patterns, in binary64."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def head_norm_rope(x, weight, eps, table, positions, sections, rot, interleaved):
    """x [T, H, D] -> (the result, the magnitudes of what was added to make it); both [T, H, D].

    Values not turned have their own magnitude.  Tokens with a position outside the table are NaN."""
    x = np.asarray(x, np.float64)
    T, H, D = x.shape
    u = x if weight is None else x / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + eps) * weight
    out, mag = u.copy(), np.abs(u)
    axis = np.repeat(np.arange(len(sections)), sections)
    for t in range(T):
        p = positions[:, t]
        if np.any(p < 0) or np.any(p >= table.shape[0]):
            out[t] = np.nan
            continue
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = float(table[p[axis[i]], i]), float(table[p[axis[i]], i + rot // 2])
            out[t, :, a] = u[t, :, a] * c - u[t, :, b] * s
            out[t, :, b] = u[t, :, b] * c + u[t, :, a] * s
            mag[t, :, a] = np.abs(u[t, :, a] * c) + np.abs(u[t, :, b] * s)
            mag[t, :, b] = np.abs(u[t, :, b] * c) + np.abs(u[t, :, a] * s)
    return out, mag


def scores(logits, kind):
    """Scores in binary64: softmax (rows of nothing but -infinity: zeros) or sigmoid.  NaN counts as -infinity,
    +infinity as the largest finite binary32 value."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return l, np.where(np.isneginf(l), 0.0, 1.0 / (1.0 + np.exp(-l)))
        e = np.where(np.isneginf(l), 0.0, np.exp(l - l.max(axis=1, keepdims=True)))
    total = e.sum(axis=1, keepdims=True)
    return l, e / np.where(total > 0, total, 1.0)


def route_grouped(logits, k, kind, bias, groups, topk_groups, group_top, renormalize, scale):
    """(ids [T, k], weights [T, k]) by sorting each token's experts."""
    l, p = scores(logits, kind)
    T, E = p.shape
    n = E // groups
    value = p if bias is None else p + np.where(np.isnan(bias), -np.inf, bias).astype(np.float64)
    choice = l if bias is None else value
    ids, weights = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        kept = range(E)
        if topk_groups < groups:
            best = []
            for g in range(groups):
                members = sorted((value[t, e] if bias is not None or group_top == 2 else l[t, e]
                                  for e in range(g * n, (g + 1) * n)), reverse=True)
                best.append((-sum(members[:group_top]), g))
            kept = [e for _, g in sorted(best)[:topk_groups] for e in range(g * n, (g + 1) * n)]
        ids[t] = [e for _, e in sorted((-choice[t, e], e) for e in kept)[:k]]
        w = p[t, ids[t]]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        weights[t] = w * scale
    return ids, weights


def dispatch(ids, E):
    """(sorted_token, expert_offsets, row_of) of the rows in the order of (expert, token, slot)."""
    T, k = ids.shape
    rows = sorted((int(ids[t, s]), t, s) for t in range(T) for s in range(k))
    sorted_token = np.array([t for _, t, _ in rows], np.int32)
    row_of = np.zeros((T, k), np.int32)
    for r, (_, t, s) in enumerate(rows):
        row_of[t, s] = r
    offsets = np.searchsorted(np.array([e for e, _, _ in rows] or [E]), np.arange(E + 1)) if T * k else np.zeros(E + 1)
    return sorted_token, offsets.astype(np.int32), row_of


def lora_add(y, x, a, b, scales, adapter, parts):
    """y [M, N], x [M, K], a [L, P R, K], b [L, N, R] -> (the result, what its rounding errors are relative to).

    The second: [M, N] sums of |t b| and, with |x| |a| in the place of t, of the products that made t."""
    y, M = np.array(y, np.float64), len(adapter)
    of_t, of_x = np.zeros_like(y), np.zeros_like(y)
    R, first = b.shape[2], np.concatenate([[0], np.cumsum(parts)])
    for m in range(M):
        e = adapter[m]
        if not 0 <= e < len(a):
            continue
        s = 1.0 if scales is None else float(scales[e])
        t, tx = s * (a[e] @ x[m]), abs(s) * (np.abs(a[e]) @ np.abs(x[m]))
        for p in range(len(parts)):
            cols, ranks = slice(first[p], first[p + 1]), slice(p * R, (p + 1) * R)
            y[m, cols] += b[e, cols] @ t[ranks]
            of_t[m, cols] = np.abs(b[e, cols]) @ np.abs(t[ranks])
            of_x[m, cols] = np.abs(b[e, cols]) @ tx[ranks]
    return y, of_t, of_x
