"""Row counts that one launch cannot hold (2^32 threads): the last rows, and those around the launches' border,
equal the call on those rows alone, bit for bit.  Narrow rows keep the tensors at a few GB."""

import pytest
import torch

import block_wise_int8_amd as bi8
from gpu_util import device

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def same(got, want):
    assert torch.equal(got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


def bands(M, per_launch):
    """Slices of rows: the first, around every launch's end, the last."""
    ends = [m for m in range(per_launch, M, per_launch)]
    return [slice(0, 40)] + [slice(m - 20, m + 20) for m in ends if m + 20 <= M] + [slice(M - 40, M)]


def hidden(M, H):
    x = torch.empty(M, H, dtype=torch.bfloat16, device=device())
    return x.normal_(generator=torch.Generator(device=device()).manual_seed(M))


@pytest.mark.parametrize("dtype", [torch.int8, F8])
def test_norm(dtype):
    M, H = (1 << 24) + 77, 9          # a workgroup of 256 threads a row
    x = hidden(M, H)
    gain = hidden(1, H)[0]
    got = bi8.rmsnorm_quant(x, gain, residual=x, dtype=dtype, return_y=True)
    for b in bands(M, 1 << 23):
        for g, w in zip(got, bi8.rmsnorm_quant(x[b], gain, residual=x[b], dtype=dtype, return_y=True)):
            same(g[b], w)


def test_quant_act():
    M, K = (1 << 26) + 77, 8          # a wave a row
    x = hidden(M, K)
    got = bi8.quant_act_fp8(x)
    for b in bands(M, 1 << 25):
        for g, w in zip(got, bi8.quant_act_fp8(x[b])):
            same(g[b], w)


def test_quant_act_gather():
    R, T, K = (1 << 26) + 77, 1000, 8
    x = hidden(T, K)
    rows = torch.randint(-1, T + 1, (R,), dtype=torch.int32, device=device())
    got = bi8.quant_act_gather_fp8(x, rows)
    for b in bands(R, 1 << 25):
        for g, w in zip(got, bi8.quant_act_gather_fp8(x, rows[b])):
            same(g[b], w)


def test_silu_mul_quant():
    R, I = (1 << 26) + 77, 16
    h = hidden(R, 2 * I)
    got = bi8.silu_mul_quant_fp8(h, return_a=True)
    for b in bands(R, 1 << 25):
        for g, w in zip(got, bi8.silu_mul_quant_fp8(h[b], return_a=True)):
            same(g[b], w)
