"""e4m3 products with nothing to round but the output, and products that split K.

Exact cases: whole codes of at most 4 and power-of-two scales.  Products of a run lie within 2^4 of each other (the
matrix core keeps 2^13), every partial sum is a multiple of 2^-2 below 2^18 and so exact in binary32, whatever the
order of its additions, and the one rounding is that to bf16: every kernel gives the same bits.

Split cases are sizes for which the library asks for a workspace: few tiles, long K, ends of K inside a block, and
columns that end inside a tile or off a 16-byte store.
"""

import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import oracle
import workloads as wl
from gpu_util import bf16_bits, bf16_to_dev, device, to_dev
from oracle import fp8
from test_gpu_fp8 import VARIANTS, check_product, codes_dev

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def whole_codes(rng, *shape):
    return fp8.encode(np.arange(-4, 5))[rng.integers(0, 9, shape)]


def scales(rng, *shape):
    return np.exp2(rng.integers(-1, 1, shape)).astype(np.float32)


def exact_case(seed, M, N, K, E=None):
    rng = np.random.default_rng(seed)
    lead = () if E is None else (E,)
    NB, KB = oracle.scale_shape(N, K)
    bias = fp8.f32_to_bf16(rng.integers(-100, 101, N).astype(np.float32))
    return (whole_codes(rng, M, K), scales(rng, M, KB), whole_codes(rng, *lead, N, K), scales(rng, *lead, NB, KB),
            bias if E is None else None)


def want_bits(ref):
    return fp8.f32_to_bf16(ref.astype(np.float32))


def gemm(xq, xs, w, ws, bias, **kw):
    return bi8.gemm_fp8(codes_dev(xq), to_dev(xs), codes_dev(w), to_dev(ws), None if bias is None else bf16_to_dev(bias),
                        **kw)


@pytest.mark.parametrize("M,N,K", [(1, 300, 144), (20, 140, 2320), (40, 260, 4112), (60, 515, 1040), (150, 270, 640),
                                   (300, 515, 2320), (520, 700, 1168)])
@pytest.mark.parametrize("variant", VARIANTS)
def test_every_variant_is_exact(M, N, K, variant):
    c = exact_case((1, M, N, K), M, N, K)
    assert np.array_equal(bf16_bits(gemm(*c, variant=variant)), want_bits(fp8.gemm_f64(*c)[0]))


@pytest.mark.parametrize("M,N,K", [(1, 300, 143), (20, 140, 2323), (40, 260, 1029), (60, 515, 131), (300, 515, 1027),
                                   (700, 1500, 403), (130, 9000, 1031)])
def test_rows_at_any_byte_are_exact(M, N, K):
    """(the last two run the tiled kernel, the others the streaming one)"""
    c = exact_case((2, M, N, K), M, N, K)
    assert np.array_equal(bf16_bits(gemm(*c)), want_bits(fp8.gemm_f64(*c)[0]))


@pytest.mark.parametrize("segments,N,K", [([0, 3, 0, 5, 0], 130, 272), ([130, 7, 260, 0, 33], 515, 1040),
                                          ([300, 1, 513], 520, 1168), ([1] * 70, 64, 144), ([2, 0, 20, 40], 140, 4112)])
@pytest.mark.parametrize("variant", [None, *VARIANTS])
def test_every_grouped_variant_is_exact(segments, N, K, variant):
    xq, xs, w, ws, _ = exact_case((3, N, K), sum(segments), N, K, len(segments))
    off = np.concatenate([[0], np.cumsum(segments)]).astype(np.int32)
    y = bi8.moe_gemm_fp8(codes_dev(xq), to_dev(xs), to_dev(off), codes_dev(w), to_dev(ws), variant=variant)
    assert np.array_equal(bf16_bits(y), want_bits(fp8.moe_gemm_f64(xq, xs, off, w, ws)[0]))


# 128 x 64 tiles, then 128 x 128; N odd, even, a multiple of 4; 2 to 8 splits; K ends inside a block in all but one
SPLIT = [(305, 211, 10832), (500, 499, 6000), (190, 82, 7840), (547, 836, 9328), (100, 2048, 8192),
         (1019, 413, 14064), (1862, 739, 14352), (1230, 456, 11552), (2822, 132, 9008)]


def split_workspace(M, N, K):
    nbytes = bi8.gemm_fp8_workspace_size(M, N, K)
    assert nbytes > 0 and nbytes % (4 * M * N) == 0 and nbytes // (4 * M * N) >= 2
    room = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device=device())   # NaN patterns
    return room, room[:nbytes]


@pytest.mark.parametrize("M,N,K", SPLIT)
def test_split_k_is_exact(M, N, K):
    """The split call equals the unsplit one and the definition bit for bit, and writes no byte past its workspace
    or its output."""
    c = exact_case((4, M, N, K), M, N, K)
    room, wsp = split_workspace(M, N, K)
    out = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=device())
    y = gemm(*c, y=out[: M * N].view(M, N), workspace=wsp)
    assert np.array_equal(bf16_bits(y), want_bits(fp8.gemm_f64(*c)[0]))
    assert torch.equal(y.view(torch.int16), gemm(*c).view(torch.int16))
    assert torch.all(room[wsp.numel():] == 0xFF) and torch.all(out[M * N:] == 7.0)
    # without a bias, into an output off the 8-byte grid
    out.fill_(7.0)
    y = gemm(*c[:4], None, y=out[1: M * N + 1].view(M, N), workspace=wsp)
    assert np.array_equal(bf16_bits(y), want_bits(fp8.gemm_f64(*c[:4])[0]))
    assert out[0] == 7.0 and torch.all(out[M * N + 1:] == 7.0)


@pytest.mark.parametrize("M,N,K", SPLIT)
@pytest.mark.parametrize("bias", [False, True])
def test_split_k(M, N, K, bias):
    rng = wl.rng_for((5, M, N, K))
    codes = lambda *s: (rng.integers(0x28, 0x60, s) | (rng.integers(0, 2, s) << 7)).astype(np.uint8)   # 2^-2 .. 30
    c = (codes(M, K), wl.weight_scales(rng, M, -(-K // 128)), codes(N, K), wl.weight_scales(rng, *oracle.scale_shape(N, K)),
         wl.activations(rng, 1, N)[0] if bias else None)
    room, wsp = split_workspace(M, N, K)
    first = gemm(*c, workspace=wsp)
    check_product(first, *fp8.gemm_f64(*c), K)
    assert torch.equal(first.view(torch.int16), gemm(*c, workspace=wsp).view(torch.int16))
    assert torch.all(room[wsp.numel():] == 0xFF)


def test_split_k_keeps_nan_codes_in_place():
    for M, N, K in ((305, 211, 10832), (1019, 413, 14064)):
        c = exact_case((6, M, N, K), M, N, K)
        xq, w = c[0], c[2]
        xq[7, K - 1], xq[M - 1, 0], w[11, K - 1], w[N - 1, K // 2] = 0x7F, 0xFF, 0x7F, 0x7F
        bad = np.zeros((M, N), bool)
        bad[[7, M - 1]], bad[:, [11, N - 1]] = True, True
        y = gemm(*c, workspace=split_workspace(M, N, K)[1])
        assert np.array_equal(np.isnan(y.float().cpu().numpy()), bad)


def test_split_k_in_a_replayed_graph():
    """Replays with other inputs, eager calls on a workspace of their own between them."""
    M, N, K = 305, 211, 10832
    cases = [exact_case((7, i), M, N, K) for i in range(3)]
    w, ws, bias = codes_dev(cases[0][2]), to_dev(cases[0][3]), bf16_to_dev(cases[0][4])
    ins = [(codes_dev(c[0]), to_dev(c[1])) for c in cases]
    xq, xs = ins[0][0].clone(), ins[0][1].clone()
    y = torch.empty(M, N, dtype=torch.bfloat16, device=device())
    wsp, own = split_workspace(M, N, K)[1], split_workspace(M, N, K)[1]
    call = lambda: bi8.gemm_fp8(xq, xs, w, ws, bias, y=y, workspace=wsp)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for r in (1, 2, 0, 1):
        xq.view(torch.uint8).copy_(ins[r][0].view(torch.uint8))
        xs.copy_(ins[r][1])
        g.replay()
        torch.cuda.synchronize()
        want = bi8.gemm_fp8(*ins[r], w, ws, bias, workspace=own)
        assert torch.equal(y.view(torch.int16), want.view(torch.int16)), "replay %d" % r


def test_streaming_kernel_past_32_bits():
    """An output of more than 2^31 elements through the streaming kernel, which the choice keeps to 64 rows: the
    last rows equal the call on those rows alone, bit for bit."""
    M, N, K, n = 262300, 8200, 128, 70
    dev = device()
    xq, w = (torch.randint(0, 120, s, dtype=torch.uint8, device=dev).view(F8) for s in ((M, K), (N, K)))
    xs, ws = torch.rand(M, 1, device=dev), torch.rand(65, 1, device=dev)
    got = bi8.gemm_fp8(xq, xs, w, ws, variant=bi8.GEMM_SKINNY)[-n:]
    want = bi8.gemm_fp8(xq[-n:], xs[-n:], w, ws, variant=bi8.GEMM_SKINNY)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
