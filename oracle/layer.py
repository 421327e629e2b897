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
