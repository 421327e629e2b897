"""Oracle of the e4m3 layer and of the normalising quantiser -- test infrastructure.

Plain numpy, written from the formats' definitions: e4m3 as a table of the 256
codes' values, rounding as a search in that table, products in binary64.
Shares no code with ``block_wise_int8_amd``.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def _table() -> np.ndarray:
    """Value of every code: sign, 4 exponent bits of bias 7, 3 mantissa bits; S.1111.111 is NaN."""
    v = np.empty(256)
    for code in range(256):
        exp, man = (code >> 3) & 15, code & 7
        mag = man / 8 * 2.0 ** -6 if exp == 0 else (1 + man / 8) * 2.0 ** (exp - 7)
        v[code] = np.nan if code & 0x7F == 0x7F else (-mag if code & 0x80 else mag)
    return v


E4M3 = _table()


def decode(codes: np.ndarray) -> np.ndarray:
    return E4M3[np.asarray(codes, np.uint8)]


def encode(q: np.ndarray) -> np.ndarray:
    """Nearest code of |q| <= 448, the even code on ties, the sign kept."""
    q = np.asarray(q, np.float64)
    a, pos = np.abs(q), E4M3[:0x7F]
    i = np.minimum(np.searchsorted(pos, a, side="right") - 1, 0x7E)
    up = np.minimum(i + 1, 0x7E)
    below, above = a - pos[i], pos[up] - a
    code = np.where((above < below) | ((above == below) & (i % 2 == 1)), up, i)
    return (code | np.where(np.signbit(q), 0x80, 0)).astype(np.uint8)


def bf16_to_f32(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def f32_to_bf16(v: np.ndarray) -> np.ndarray:
    """Round binary32 to the nearest bf16, ties to even (finite values)."""
    u = np.ascontiguousarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def _scales(amax: np.ndarray, top: float) -> np.ndarray:
    return amax.astype(np.float32) / np.float32(top)


def _quotient(v: np.ndarray, s: np.ndarray) -> np.ndarray:
    """The binary32 quotient v / s, 0 where s is 0."""
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(s > 0, v / s, np.float32(0)).astype(np.float32)


def quant_f32(v: np.ndarray, fp8: bool = True, group: int = 128):
    """Codes (uint8 or int8) and scales of fp32 values [M, K], groups of `group` columns."""
    M, K = v.shape
    top = E4M3_MAX if fp8 else 127.0
    KB = -(-K // group)
    pad = np.zeros((M, KB * group), np.float32)
    pad[:, :K] = v
    s = _scales(np.abs(pad).reshape(M, KB, group).max(-1), top)
    q = np.clip(_quotient(pad.reshape(M, KB, group), s[..., None]), -top, top)
    codes = encode(q) if fp8 else np.rint(q).astype(np.int8)
    return codes.reshape(M, KB * group)[:, :K].copy(), s


def quant_act(x_bits: np.ndarray):
    return quant_f32(bf16_to_f32(x_bits))


def quant_weight(w_bits: np.ndarray):
    """One scale per 128 x 128 block: (codes [N, K], scales [ceil(N/128), ceil(K/128)])."""
    w = bf16_to_f32(w_bits)
    N, K = w.shape
    NB, KB = -(-N // 128), -(-K // 128)
    pad = np.zeros((NB * 128, KB * 128), np.float32)
    pad[:N, :K] = w
    s = _scales(np.abs(pad).reshape(NB, 128, KB, 128).max((1, 3)), E4M3_MAX)
    q = _quotient(pad, s.repeat(128, 0).repeat(128, 1))
    return encode(np.clip(q, -E4M3_MAX, E4M3_MAX))[:N, :K].copy(), s


def _peaks(v: np.ndarray) -> np.ndarray:
    """The largest absolute value of every eight consecutive columns."""
    M, K = v.shape
    pad = np.zeros((M, -(-K // 8) * 8))
    pad[:, :K] = np.abs(v)
    return pad.reshape(M, pad.shape[1] // 8, 8).max(-1)


def gemm_f64(xq, xs, w, ws, bias_bits=None):
    """(y, mag, peak) in binary64, before the rounding to bf16: mag is the sum of the absolute terms, peak a
    bound on the sum, over runs of eight consecutive columns, of the largest absolute term."""
    K, N = xq.shape[1], w.shape[0]
    x = decode(xq) * np.asarray(xs, np.float64).repeat(128, 1)[:, :K]
    wd = decode(w) * np.asarray(ws, np.float64).repeat(128, 0)[:N].repeat(128, 1)[:, :K]
    y, mag, peak = x @ wd.T, np.abs(x) @ np.abs(wd).T, _peaks(x) @ _peaks(wd).T
    if bias_bits is not None:
        b = bf16_to_f32(bias_bits).astype(np.float64)
        y, mag = y + b, mag + np.abs(b)
    return y, mag, peak


def moe_gemm_f64(xq, xs, offsets, w, ws):
    parts = [gemm_f64(xq[a:b], xs[a:b], w[e], ws[e]) for e, (a, b) in enumerate(zip(offsets, offsets[1:]))]
    return tuple(np.concatenate(p) for p in zip(*parts))


def rmsnorm(x_bits, weight_bits, eps: float, residual_bits=None, fp8: bool = False):
    """(codes, scales, h bf16 bits, y fp32): the row's norm, quantised."""
    h_bits = x_bits if residual_bits is None else f32_to_bf16(bf16_to_f32(x_bits) + bf16_to_f32(residual_bits))
    h = bf16_to_f32(h_bits)
    mean = np.square(h.astype(np.float64)).sum(-1, keepdims=True) / h.shape[1]
    rstd = (1.0 / np.sqrt(mean + eps)).astype(np.float32)
    y = (h * rstd) * bf16_to_f32(weight_bits)
    codes, s = quant_f32(y, fp8)
    return codes, s, h_bits, y
