"""Pins of the e4m3 oracle (no GPU): the format against torch's conversions and closed forms."""
import numpy as np
import pytest
import torch

import workloads as wl
from oracle import fp8


def test_table_is_the_format():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.E4M3, v, equal_nan=True)
    assert fp8.E4M3[0x7E] == 448 and fp8.E4M3[0x08] == 2.0 ** -6 and fp8.E4M3[0x01] == 2.0 ** -9


def test_encode_is_the_inverse_and_rounds_ties_to_even():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    assert np.array_equal(fp8.encode(fp8.decode(codes)), codes)
    pos = fp8.E4M3[:0x7F]
    mid = (pos[1:] + pos[:-1]) / 2
    got = fp8.encode(mid)
    assert np.all(got % 2 == 0) and np.all((got == np.arange(126)) | (got == np.arange(1, 127)))


def test_encode_agrees_with_torch():
    rng = np.random.default_rng(3)
    v = (rng.standard_normal(200000) * np.exp2(rng.uniform(-14, 9, 200000))).astype(np.float32).clip(-448, 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(v), want)


def test_quantiser_invariants():
    x = wl.activations(np.random.default_rng(4), 9, 300, 0.05)
    q, s = fp8.quant_act(x)
    v, xf = fp8.decode(q), fp8.bf16_to_f32(x)
    assert s.shape == (9, 3) and np.abs(v).max() == 448
    full = s.repeat(128, 1)[:, :300].astype(np.float64)
    # half a step of e4m3 (2^-4 relative, 2^-10 in the subnormals) and the quotient's rounding
    assert np.all(np.abs(v * full - xf) <= full * (np.abs(xf) / full * (2.0 ** -4 + 2.0 ** -22) + 2.0 ** -10))
    z, sz = fp8.quant_act(np.zeros((2, 130), np.uint16))
    assert not z.any() and not sz.any()


def test_weight_blocks_and_product():
    rng = np.random.default_rng(5)
    w = wl.activations(rng, 200, 300)
    q, s = fp8.quant_weight(w)
    assert s.shape == (2, 3)
    blk, sb = fp8.quant_weight(w[128:, 128:256])
    assert np.array_equal(q[128:, 128:256], blk) and s[1, 1] == sb[0, 0]
    xq, xs = fp8.quant_act(wl.activations(rng, 3, 300))
    y, mag, peak = fp8.gemm_f64(xq, xs, q, s)
    assert np.all(np.abs(y) <= mag) and np.all(peak <= mag * 8) and np.all(8 * peak >= mag)
    brute = sum(fp8.E4M3[xq[1, k]] * fp8.E4M3[q[150, k]] * float(xs[1, k // 128]) * float(s[1, k // 128])
                for k in range(300))
    assert abs(y[1, 150] - brute) <= 1e-12 * mag[1, 150]


@pytest.mark.parametrize("fp8_codes", [False, True])
def test_rmsnorm_against_its_formula(fp8_codes):
    rng = np.random.default_rng(6)
    x, r, g = wl.activations(rng, 5, 200), wl.activations(rng, 5, 200), wl.activations(rng, 1, 200)[0]
    q, s, h, y = fp8.rmsnorm(x, g, 1e-5, r, fp8_codes)
    hs = (torch.from_numpy(x.view(np.int16)).view(torch.bfloat16) + torch.from_numpy(r.view(np.int16)).view(torch.bfloat16))
    assert np.array_equal(hs.view(torch.int16).numpy().view(np.uint16), h)
    hd = fp8.bf16_to_f32(h).astype(np.float64)
    want = hd / np.sqrt((hd ** 2).mean(1, keepdims=True) + 1e-5) * fp8.bf16_to_f32(g)
    # three roundings to binary32: rstd and the two products
    assert np.all(np.abs(y - want) <= np.abs(want) * 3 * 2.0 ** -24 * 1.001)
    assert s.shape == (5, 2)
    assert np.array_equal(q, fp8.quant_f32(y, fp8_codes)[0])
