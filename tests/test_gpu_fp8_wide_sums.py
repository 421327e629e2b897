"""The e4m3 products whose sums binary32 holds: the streaming kernel, GEMM_TILE_256X128_F16, and the layer's w13
where it runs them.

Exact cases hold what the f8 matrix instruction cuts off: runs of eight with products of 2^16 that cancel and others
of 2^-2 to 2^4 that remain.  Every partial sum, in any order, is a multiple of 2^-2 below 2^22 (128 products of a
block of at most 2^16, the blocks' sums small) and so exact in binary32: the result is the definition's bit for bit.
"""

import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import oracle
from gpu_util import bf16_bits, bf16_to_dev, device, to_dev
from oracle import fp8
from test_gpu_fp8 import check_product, codes_dev, grouped_case, product_case, run_grouped
from test_gpu_fp8_layer import layer_case, scratch, stages

pytestmark = pytest.mark.gpu

F16 = bi8.GEMM_TILE_256X128_F16
HOLD = [bi8.GEMM_SKINNY, F16]


def cancelling(rng, M, N, K):
    """Codes [M, K] and [N, K]: of every eight, two places hold 256 and +-256 against 256 and -+256, the others
    +-0.5 to +-4."""
    values = np.array([0.5, 1, 1.5, 2, 3, 4])
    x, w = (values[rng.integers(0, 6, s)] * rng.choice([-1, 1], s) for s in ((M, K), (N, K)))
    x[:, 0::8], x[:, 5::8] = 256, 256
    w[:, 0::8], w[:, 5::8] = 256, -256
    return x, w


def exact_case(seed, M, N, K, E=None):
    rng = np.random.default_rng(seed)
    x, w = cancelling(rng, M, N * (E or 1), K)
    # (K % 8 == 0: the big products of a run cancel, whatever the order)
    w = fp8.encode(w).reshape((N, K) if E is None else (E, N, K))
    NB, KB = oracle.scale_shape(N, K)
    return fp8.encode(x), np.ones((M, KB), np.float32), w, np.ones(((E,) if E else ()) + (NB, KB), np.float32)


def want_bits(ref):
    return fp8.f32_to_bf16(ref.astype(np.float32))


def gemm(xq, xs, w, ws, bias=None, **kw):
    return bi8.gemm_fp8(codes_dev(xq), to_dev(xs), codes_dev(w), to_dev(ws), None if bias is None else bf16_to_dev(bias),
                        **kw)


@pytest.mark.parametrize("variant", HOLD)
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (3, 260, 112), (20, 100, 4096), (40, 140, 1040), (65, 129, 128),
                                   (130, 300, 272), (257, 515, 1040), (520, 700, 144), (300, 1030, 2320)])
def test_dense(M, N, K, variant):
    c = exact_case((1, M, N, K), M, N, K)
    assert np.array_equal(bf16_bits(gemm(*c, variant=variant)), want_bits(fp8.gemm_f64(*c)[0]))
    c = product_case((2, M, N, K), M, N, K, True)
    check_product(gemm(*c, variant=variant), *fp8.gemm_f64(*c), K)


@pytest.mark.parametrize("M", [31, 32, 33, 63, 64, 66, 95, 96, 97, 128, 160, 161])
def test_sub_rows_without_rows(M):
    """The F16 tiles leave out 32-row sub-rows that have no rows: tiles that end on both sides of each."""
    N, K = 300, 400
    c = exact_case((8, M), M, N, K)
    room = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=device())
    y = gemm(*c, variant=F16, y=room[: M * N].view(M, N))
    assert np.array_equal(bf16_bits(y), want_bits(fp8.gemm_f64(*c)[0])) and torch.all(room[M * N:] == 7.0)


@pytest.mark.parametrize("M,N,K", [(1, 40, 24), (9, 100, 1000), (30, 260, 136), (70, 300, 4104)])
def test_streamed_rows_off_the_16_byte_grid(M, N, K):
    c = exact_case((7, M, N, K), M, N, K)
    assert bi8.gemm_fp8_select(M, N, K) == bi8.GEMM_SKINNY
    assert np.array_equal(bf16_bits(gemm(*c)), want_bits(fp8.gemm_f64(*c)[0]))


def test_the_cut_that_it_avoids():
    """(pins what the header says of the other kernels: beside 2^16 they drop products below 2^3)"""
    x, w = np.zeros((1, 128)), np.zeros((1, 128))
    x[0, :8], w[0, :8] = [256, 2, 2, 2, 2, 256, 2, 2], [256, 1, 1, 1, 1, -256, 1, 1]
    c = fp8.encode(x), np.ones((1, 1), np.float32), fp8.encode(w), np.ones((1, 1), np.float32)
    for v in (None, *HOLD):
        assert gemm(*c, variant=v).item() == 12.0
    assert gemm(*c, variant=bi8.GEMM_TILE_256X128).item() == 0.0


@pytest.mark.parametrize("segments,N,K", [([1], 16, 16), ([0, 3, 0, 5, 0], 130, 272), ([130, 7, 260, 0, 33], 640, 272),
                                          ([300, 1, 513], 520, 1168), ([1] * 70, 64, 144)])
@pytest.mark.parametrize("variant", HOLD)
def test_grouped(segments, N, K, variant):
    xq, xs, w, ws = exact_case((3, N, K), sum(segments), N, K, len(segments))
    off = np.concatenate([[0], np.cumsum(segments)]).astype(np.int32)
    y = run_grouped(xq, xs, off, w, ws, variant=variant)
    assert np.array_equal(bf16_bits(y), want_bits(fp8.moe_gemm_f64(xq, xs, off, w, ws)[0]))
    c = grouped_case((4, N, K), segments, N, K)
    check_product(run_grouped(*c, variant=variant), *fp8.moe_gemm_f64(*c), K)
    # rows behind the last segment stay
    n = sum(segments)
    off = off.copy()
    off[off > n - 1] = n - 1
    y = torch.full((n, N), 5.0, dtype=torch.bfloat16, device=device())
    run_grouped(xq, xs, off, w, ws, variant=variant, y=y)
    assert torch.all(y[n - 1:] == 5.0)


def test_nan_codes_stay_in_place_and_long_k():
    M, N, K = 300, 290, 400
    xq, xs, w, ws, _ = product_case((5, M, N, K), M, N, K, False)
    xq[7, K - 1], xq[299, 0], w[11, K - 1], w[289, 0] = 0x7F, 0xFF, 0x7F, 0x7F
    bad = np.zeros((M, N), bool)
    bad[[7, 299]], bad[:, [11, 289]] = True, True
    assert np.array_equal(np.isnan(gemm(xq, xs, w, ws, variant=F16).float().cpu().numpy()), bad)
    c = product_case((6,), 300, 260, 66000, False)
    check_product(gemm(*c, variant=F16), *fp8.gemm_f64(*c), 66000)


def wide_stages(x, logits, w13, s13, w2, s2, k):
    """The layer by its separate calls, w13 by the F16 variant."""
    T, H = x.shape
    E, N, _ = w13.shape
    _, weights, order, off, row_of = bi8.moe_route(logits, k)
    xq, xs = bi8.quant_act_gather_fp8(x, order)
    aq, as_ = bi8.silu_mul_quant_fp8(bi8.moe_gemm_fp8(xq, xs, off, w13, s13, variant=F16))
    n2 = bi8.moe_gemm_fp8_workspace_size(T * k, H, N // 2, E)
    return bi8.moe_combine(bi8.moe_gemm_fp8(aq, as_, off, w2, s2, workspace=scratch(n2)), row_of, weights)


LAYERS = [(1, 2, 128, 128, 1), (3, 8, 256, 144, 2), (40, 3, 384, 256, 2), (257, 5, 256, 400, 4), (700, 4, 512, 640, 2),
          (100, 2, 1024, 4096, 1), (62, 3, 3456, 128, 2), (227, 2, 3456, 544, 1), (8, 64, 512, 256, 8)]


@pytest.mark.parametrize("T,E,H,I,k", LAYERS)
def test_layer_is_its_stages(T, E, H, I, k):
    d = layer_case(31 + T, T, E, H, I)
    want = wide_stages(*d, k)
    nbytes = bi8.moe_layer_fp8_workspace_size(T, H, I, E, k)
    room = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device=device())
    for _ in range(2):
        got = bi8.moe_layer_fp8(*d, k, workspace=room[:nbytes], variant=F16)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert torch.all(room[nbytes:] == 0xFF)


def test_layer_in_a_replayed_graph():
    T, E, H, I, k = 90, 4, 512, 384, 2
    cases = [layer_case(51 + r, T, E, H, I) for r in range(3)]
    w = cases[0][2:]
    x, logits, out = cases[0][0].clone(), cases[0][1].clone(), torch.empty_like(cases[0][0])
    wsp = scratch(bi8.moe_layer_fp8_workspace_size(T, H, I, E, k))
    call = lambda: bi8.moe_layer_fp8(x, logits, *w, k, out=out, workspace=wsp, variant=F16)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for r in (1, 2, 0, 1):
        x.copy_(cases[r][0])
        logits.copy_(cases[r][1])
        g.replay()
        torch.cuda.synchronize()
        want = wide_stages(cases[r][0], cases[r][1], *w, k)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), "replay %d" % r


# (T, E, H, I, k), what the layer runs for w13 by itself: weights of 60 MB and more, rows enough for tiles
@pytest.mark.parametrize("T,E,H,I,k,w13", [(256, 64, 2048, 1024, 8, F16), (256, 64, 2048, 1008, 8, F16),
                                           (40, 64, 2048, 1024, 8, bi8.GEMM_SKINNY), (3, 8, 1024, 512, 2, bi8.GEMM_SKINNY)])
def test_layer_holds_its_sums_where_the_weights_bound_it(T, E, H, I, k, w13):
    assert bi8.moe_layer_fp8_select(T, H, I, E, k) == w13
    d = layer_case(61, T, E, H, I)
    want = stages(*d, k)[0]
    nbytes = bi8.moe_layer_fp8_workspace_size(T, H, I, E, k)
    room = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device=device())
    for kw in (dict(workspace=room[:nbytes]), {}):
        assert torch.equal(bi8.moe_layer_fp8(*d, k, **kw).view(torch.int16), want.view(torch.int16))
    assert torch.all(room[nbytes:] == 0xFF)
    if w13 == F16:
        assert torch.equal(bi8.moe_layer_fp8(*d, k, variant=F16).view(torch.int16), want.view(torch.int16))


def test_layer_refuses_other_variants():
    d = layer_case(1, 4, 2, 128, 128)
    for v in (-1, bi8.GEMM_SKINNY, bi8.GEMM_TILE_256X128, 6, 9):
        with pytest.raises(bi8.BlockInt8Error, match="variant"):
            bi8.moe_layer_fp8(*d, 1, variant=v)
