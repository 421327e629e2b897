"""The e4m3 MoE layer where its grouped products split K on the layer's workspace, and in its decoding form with
many experts: bit for bit with its stages, each called on its own."""

import pytest
import torch

import block_wise_int8_amd as bi8
from gpu_util import device

pytestmark = pytest.mark.gpu


def scratch(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device=device()) if nbytes else None


def stages(x, logits, w13, s13, w2, s2, k, renormalize=False):
    """The layer by its separate calls, each grouped product with the workspace it asks for; and those sizes."""
    T, H = x.shape
    E, N, _ = w13.shape
    I = N // 2
    _, weights, order, off, row_of = bi8.moe_route(logits, k, renormalize)
    xq, xs = bi8.quant_act_gather_fp8(x, order)
    n13, w13_runs = 0, bi8.moe_layer_fp8_select(T, H, I, E, k)
    if I % 128 == 0 and w13_runs in (bi8.GEMM_TILE_256X128, bi8.GEMM_TILE_256X256):
        aq, as_ = bi8.moe_gemm_silu_quant_fp8(xq, xs, off, w13, s13)
    elif w13_runs in (bi8.GEMM_SKINNY, bi8.GEMM_TILE_256X128_F16):
        aq, as_ = bi8.silu_mul_quant_fp8(bi8.moe_gemm_fp8(xq, xs, off, w13, s13, variant=w13_runs))
    else:
        n13 = bi8.moe_gemm_fp8_workspace_size(T * k, N, H, E)
        aq, as_ = bi8.silu_mul_quant_fp8(bi8.moe_gemm_fp8(xq, xs, off, w13, s13, workspace=scratch(n13)))
    n2 = bi8.moe_gemm_fp8_workspace_size(T * k, H, I, E)
    y2 = bi8.moe_gemm_fp8(aq, as_, off, w2, s2, workspace=scratch(n2))
    return bi8.moe_combine(y2, row_of, weights), n13, n2


def layer_case(seed, T, E, H, I):
    """(x, logits, w13, its scales, w2, its scales), codes of 2^-2 to 30."""
    g = torch.Generator(device=device()).manual_seed(seed)
    blocks = lambda n: -(-n // 128)

    def codes(*shape):
        sign = torch.randint(0, 2, shape, dtype=torch.uint8, device=device(), generator=g) << 7
        c = torch.randint(0x28, 0x60, shape, dtype=torch.uint8, device=device(), generator=g)
        return (c | sign).view(torch.float8_e4m3fn)

    def scales(*shape):
        return 0.002 + 0.002 * torch.rand(*shape, device=device(), generator=g)

    x = torch.randn(T, H, device=device(), generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, device=device(), generator=g)
    return (x, logits, codes(E, 2 * I, H), scales(E, blocks(2 * I), blocks(H)), codes(E, H, I),
            scales(E, blocks(H), blocks(I)))


# (T, E, H, I, k), which product splits K
SPLIT = [(100, 2, 1024, 4096, 1, "w2"), (62, 3, 3456, 128, 2, ""), (227, 2, 3456, 544, 1, "w13"),
         (42, 1, 5600, 3280, 1, "w13 w2"), (1, 64, 1024, 384, 8, ""), (8, 256, 512, 256, 8, ""), (3, 130, 256, 400, 2, "")]


@pytest.mark.parametrize("T,E,H,I,k,split", SPLIT)
def test_layer_is_its_stages(T, E, H, I, k, split):
    d = layer_case(91 + T, T, E, H, I)
    for renormalize in (False, True):
        want, n13, n2 = stages(*d, k, renormalize)
        assert (n13 > 0, n2 > 0) == ("w13" in split, "w2" in split)
        nbytes = bi8.moe_layer_fp8_workspace_size(T, H, I, E, k)
        assert nbytes >= max(n13, n2)
        room = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device=device())   # NaN patterns
        for _ in range(2):
            got = bi8.moe_layer_fp8(*d, k, renormalize, workspace=room[:nbytes])
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert torch.all(room[nbytes:] == 0xFF)
        assert torch.equal(bi8.moe_layer_fp8(*d, k, renormalize).view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T,E,H,I,k", [(100, 2, 1024, 4096, 1), (227, 2, 3456, 544, 1), (1, 64, 1024, 384, 8)])
def test_layer_in_a_replayed_graph(T, E, H, I, k):
    cases = [layer_case(92 + r, T, E, H, I) for r in range(3)]
    w, nbytes = cases[0][2:], bi8.moe_layer_fp8_workspace_size(T, H, I, E, k)
    x, logits = cases[0][0].clone(), cases[0][1].clone()
    out, wsp = torch.empty_like(x), torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=device())
    call = lambda: bi8.moe_layer_fp8(x, logits, *w, k, out=out, workspace=wsp)
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
        want = stages(cases[r][0], cases[r][1], *w, k)[0]
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), "replay %d" % r
