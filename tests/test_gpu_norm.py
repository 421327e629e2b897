"""The normalising quantiser on the GPU against its oracle: codes, scales and the sum bit for bit (the
definition fixes every rounding but the order of a binary64 sum), y to half a step of bf16."""
import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import oracle
import workloads as wl
from gpu_util import assert_gemm_close, bf16_bits, bf16_to_dev, bits_to_f64, device, to_dev
from oracle import fp8
from test_gpu_fp8 import check_product

pytestmark = pytest.mark.gpu

EPS = 1e-6


def gain(rng, H):
    return wl.to_bf16_bits((1 + 0.1 * rng.standard_normal(H)).astype(np.float32))


def check(x, g, r, is_fp8, out, eps=EPS):
    """out: (xq, xs[, h], y) of the call on bits x, gain bits g, residual bits r."""
    q, s, h, y = fp8.rmsnorm(x, g, eps, r, is_fp8)
    xq, xs = out[0], out[1].cpu().numpy()
    assert np.array_equal(xs, s)
    got = xq.view(torch.uint8).cpu().numpy().view(q.dtype)
    zero = (s == 0).repeat(128, 1)[:, : got.shape[1]]
    assert np.array_equal(got, np.where(zero, 0, q))
    if r is not None:
        assert np.array_equal(bf16_bits(out[2]), h)
    yb = bits_to_f64(bf16_bits(out[-1]))
    assert np.all(np.abs(yb - y) <= np.abs(y.astype(np.float64)) * 2.0 ** -8 + 2.0 ** -134)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("M,H,residual,pad", [
    (1, 1, False, 0), (1, 8, True, 0), (3, 7, True, 0), (2, 128, True, 0), (5, 200, False, 0), (4, 136, True, 8),
    (9, 1000, True, 24), (1, 4096, True, 0), (7, 4000, False, 96), (3, 4001, True, 0), (6, 2048, True, 3),
    (130, 5120, True, 0), (33, 8192, True, 0), (5, 14336, False, 0), (2, 16392, True, 0), (2, 20000, False, 8),
    (2050, 512, True, 0), (4099, 1536, True, 0), (2049, 4096, False, 0), (2500, 264, True, 0), (2, 9001, True, 0)])
def test_rmsnorm_quant(M, H, residual, pad, dtype):
    rng = wl.rng_for((91, M, H))
    x, g = wl.activations(rng, M, H + pad, 0.01), gain(rng, H)
    r = wl.activations(rng, M, H + pad, 0.01) if residual else None
    xd, rd = bf16_to_dev(x)[:, :H], None if r is None else bf16_to_dev(r)[:, :H]
    out = bi8.rmsnorm_quant(xd, bf16_to_dev(g), EPS, rd, dtype=dtype, return_y=True)
    assert len(out) == (4 if residual else 3)
    x = np.ascontiguousarray(x[:, :H])
    check(x, g, None if r is None else np.ascontiguousarray(r[:, :H]), dtype != torch.int8, out)
    # without the bf16 output the others are the same
    again = bi8.rmsnorm_quant(xd, bf16_to_dev(g), EPS, rd, dtype=dtype)
    for a, b in zip(again, out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("H", [256, 4096, 4001, 20000])
@pytest.mark.parametrize("place", ["x", "residual"])
def test_sum_in_place(H, place):
    rng = wl.rng_for((92, H))
    x, r, g = wl.activations(rng, 6, H), wl.activations(rng, 6, H), gain(rng, H)
    xd, rd = bf16_to_dev(x), bf16_to_dev(r)
    out = bi8.rmsnorm_quant(xd, bf16_to_dev(g), EPS, rd, h=xd if place == "x" else rd, return_y=True)
    check(x, g, r, False, out)
    assert out[2].data_ptr() == (xd if place == "x" else rd).data_ptr()


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_special_rows(dtype):
    rng = wl.rng_for(93)
    H = 384
    x, g = wl.activations(rng, 7, H), gain(rng, H)
    x[1] = 0                                                     # a row of zeros
    x[2] = wl.to_bf16_bits(np.full(H, 1e30, np.float32))         # squares past binary32
    x[3] = wl.to_bf16_bits(np.full(H, 1e-30, np.float32))        # eps decides
    x[4, :128] = 0                                               # one group of zeros
    x[5, 200] = 0x7FC0                                           # NaN
    g[7] = 0
    out = bi8.rmsnorm_quant(bf16_to_dev(x), bf16_to_dev(g), EPS, dtype=dtype, return_y=True)
    keep = [0, 1, 2, 3, 4, 6]
    check(x[keep], g, None, dtype != torch.int8, tuple(t[keep] for t in out))
    assert torch.isnan(out[1][5]).all()
    zeros = bi8.rmsnorm_quant(bf16_to_dev(x[1:2]), bf16_to_dev(g), 0.0, dtype=dtype)
    assert torch.isnan(zeros[1]).all()


def test_large_rows_of_ones_are_exact():
    """rstd = 1 for a row of ones without eps: the codes are the weight's own, for any length."""
    for H in (128, 8192, 30000, 65536):
        w = wl.to_bf16_bits(np.linspace(-2, 2, H).astype(np.float32))
        q, s = bi8.rmsnorm_quant(bf16_to_dev(np.full((2, H), 0x3F80, np.uint16)), bf16_to_dev(w), 0.0)
        want_q, want_s = fp8.quant_f32(fp8.bf16_to_f32(np.stack([w, w])), False)
        assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_norm_feeds_the_linear(dtype):
    """The run they are made for: residual, norm, projection."""
    rng = wl.rng_for(94)
    M, H, N = 37, 640, 300
    x, r, g, wb = wl.activations(rng, M, H), wl.activations(rng, M, H), gain(rng, H), wl.activations(rng, N, H)
    xq, xs, h = bi8.rmsnorm_quant(bf16_to_dev(x), bf16_to_dev(g), EPS, bf16_to_dev(r), dtype=dtype)
    q, s, hb, _ = fp8.rmsnorm(x, g, EPS, r, dtype != torch.int8)
    assert np.array_equal(bf16_bits(h), hb)
    if dtype == torch.int8:
        wq, ws = bi8.quant_weight(bf16_to_dev(wb))
        assert_gemm_close(bf16_bits(bi8.gemm(xq, xs, wq, ws)), oracle.gemm(q, s, *oracle.quant_weight(wb)), "int8")
    else:
        wq, ws = bi8.quant_weight_fp8(bf16_to_dev(wb))
        check_product(bi8.gemm_fp8(xq, xs, wq, ws), *fp8.gemm_f64(q, s, *fp8.quant_weight(wb)), H)


def test_replays_equal_eager():
    rng = wl.rng_for(95)
    M, H = 20, 1024
    ins = [(bf16_to_dev(wl.activations(rng, M, H)), bf16_to_dev(wl.activations(rng, M, H))) for _ in range(3)]
    g = bf16_to_dev(gain(rng, H))
    x, r = ins[0][0].clone(), ins[0][1].clone()
    xq, xs, h, y = bi8.rmsnorm_quant(x, g, EPS, r, return_y=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bi8.rmsnorm_quant(x, g, EPS, r, xq=xq, xs=xs, h=h, y=y)
    for a, b in ins:
        x.copy_(a)
        r.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip((xq, xs, h, y), bi8.rmsnorm_quant(a, g, EPS, b, return_y=True)):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def test_binding_refusals():
    dev = device()
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=dev)
    w = x[0].clone()
    bad = [
        (TypeError, lambda: bi8.rmsnorm_quant(x.float(), w)),
        (TypeError, lambda: bi8.rmsnorm_quant(x, w.float())),
        (ValueError, lambda: bi8.rmsnorm_quant(x, w[:128])),
        (TypeError, lambda: bi8.rmsnorm_quant(x, w, dtype=torch.float16)),
        (ValueError, lambda: bi8.rmsnorm_quant(x, w, residual=x[:2])),
        (ValueError, lambda: bi8.rmsnorm_quant(x, w, h=x)),
        (ValueError, lambda: bi8.rmsnorm_quant(x, w, residual=x, h=x.t())),
        (ValueError, lambda: bi8.rmsnorm_quant(x, w, y=x[:2])),
        (ValueError, lambda: bi8.rmsnorm_quant(x, w.cpu())),
        (bi8.BlockInt8Error, lambda: bi8.rmsnorm_quant(x, w, eps=-1.0)),
    ]
    for error, fn in bad:
        with pytest.raises(error):
            fn()
    assert bi8.rmsnorm_quant(x[:0], w)[0].shape == (0, 256)
