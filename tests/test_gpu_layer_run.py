"""A run of the operators beside the 8-bit products as a served layer makes it: norm, int8 query / key / value
projection with adapters, head norm and rotation, then norm, router and experts.  Each step is compared with the oracle
on what the step before gave; then the whole run is captured, replayed on other inputs and on another stream."""
import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import workloads as wl
from gpu_util import bf16_bits, bf16_to_dev, device, to_dev
from oracle import layer
from test_gpu_heads import check as check_heads
from test_gpu_heads import rope_table
from test_gpu_lora import check as check_lora
from test_gpu_route import check as check_route

pytestmark = pytest.mark.gpu

H, HQ, HK, D, R, L, E, K, I = 256, 4, 2, 64, 8, 3, 16, 4, 128
PARTS = (HQ * D, HK * D, HK * D)
N = sum(PARTS)
ROUTE = dict(score="sigmoid", groups=4, topk_groups=2, group_top=2, renormalize=True, scale=2.0)


class Layer:
    """The weights, and the workspaces of one caller."""

    def __init__(self, rng, T):
        gain = lambda n: bf16_to_dev(wl.to_bf16_bits((1 + 0.1 * rng.standard_normal(n)).astype(np.float32)))
        self.gain1, self.gain2, self.q_gain, self.k_gain = gain(H), gain(H), gain(D), gain(D)
        self.w, self.ws = to_dev(wl.weights(rng, N, H)), to_dev(wl.weight_scales(rng, *bi8.scale_shape(N, H)))
        self.a = bf16_to_dev(wl.to_bf16_bits((rng.standard_normal((L, 3 * R, H)) / 16).astype(np.float32)))
        self.b = bf16_to_dev(wl.to_bf16_bits((rng.standard_normal((L, N, R)) / 3).astype(np.float32)))
        self.scales = to_dev(rng.uniform(0.5, 2, L).astype(np.float32))
        self.table = to_dev(rope_table(64, D))
        self.router = to_dev((rng.standard_normal((E, H)) / 16).astype(np.float32))
        self.bias = to_dev((0.1 * rng.standard_normal(E)).astype(np.float32))
        q = [bi8.quant_weight_fp8(bf16_to_dev(wl.activations(rng, 2 * I, H))) for _ in range(E)]
        self.w13, self.ws13 = torch.stack([w.view(torch.uint8) for w, _ in q]).view(torch.float8_e4m3fn), torch.stack([s for _, s in q])
        q = [bi8.quant_weight_fp8(bf16_to_dev(wl.activations(rng, H, I))) for _ in range(E)]
        self.w2, self.ws2 = torch.stack([w.view(torch.uint8) for w, _ in q]).view(torch.float8_e4m3fn), torch.stack([s for _, s in q])
        sizes = (bi8.lora_add_workspace_size(T, H, R, 3), bi8.moe_route_grouped_workspace_size(T, E),
                 bi8.moe_layer_fp8_workspace_size(T, H, I, E, K, routed=True))
        self.scratch = [torch.empty(max(n, 16), dtype=torch.uint8, device=device()) for n in sizes]

    def run(self, x, residual, adapter, positions, check=False):
        T = x.shape[0]
        xq, xs, h, y = bi8.rmsnorm_quant(x, self.gain1, residual=residual, return_y=True)
        qkv = bi8.gemm(xq, xs, self.w, self.ws)
        plain = qkv.clone()
        bi8.lora_add(qkv, y, self.a, self.b, adapter, self.scales, PARTS, self.scratch[0])
        heads = qkv.view(T, HQ + 2 * HK, D)
        before = qkv.clone().view_as(heads)
        q, k = bi8.qk_norm_rope(heads[:, :HQ], heads[:, HQ: HQ + HK], positions, self.table, self.q_gain, self.k_gain,
                                sections=(16, 8, 8), q_out=heads[:, :HQ], k_out=heads[:, HQ: HQ + HK])
        xq, xs, h2, y2 = bi8.rmsnorm_quant(qkv[:, :H], self.gain2, residual=h, return_y=True)
        logits = y2.float() @ self.router.t()
        route = bi8.moe_route_grouped(logits, K, bias=self.bias, workspace=self.scratch[1], **ROUTE)
        out = bi8.moe_layer_fp8(y2, None, self.w13, self.ws13, self.w2, self.ws2, K, route=route, workspace=self.scratch[2])
        if check:
            b = lambda t: bf16_bits(t.contiguous())
            check_lora(b(before.view(T, N)), b(y), b(self.a), b(self.b), b(plain), self.scales.cpu().numpy(),
                       adapter.cpu().numpy(), PARTS)
            tab, pos = self.table.cpu().numpy(), positions.cpu().numpy()
            check_heads(b(q), b(before[:, :HQ]), b(self.q_gain), tab, pos, (16, 8, 8), D, False)
            check_heads(b(k), b(before[:, HQ: HQ + HK]), b(self.k_gain), tab, pos, (16, 8, 8), D, False)
            assert torch.equal(heads[:, HQ + HK:], before[:, HQ + HK:])
            check_route(route, logits.cpu().numpy().astype(np.float64), K, bias=self.bias.cpu().numpy(), **ROUTE)
            assert torch.equal(out, bi8.moe_layer_fp8(y2, None, self.w13, self.ws13, self.w2, self.ws2, K, route=route))
        return out, qkv, route[3]


def inputs(rng, T):
    return (bf16_to_dev(wl.activations(rng, T, H)), bf16_to_dev(wl.activations(rng, T, H)),
            to_dev(rng.integers(-1, L, T).astype(np.int32)), to_dev(rng.integers(0, 64, (3, T)).astype(np.int32)))


@pytest.mark.parametrize("T", [1, 37, 300])
def test_the_run(T):
    rng = wl.rng_for((131, T))
    Layer(rng, T).run(*inputs(rng, T), check=True)


@pytest.mark.parametrize("T", [3, 90])
def test_captured_replayed_and_on_two_streams(T):
    rng = wl.rng_for((132, T))
    one = Layer(rng, T)
    sets = [inputs(rng, T) for _ in range(4)]
    held = [t.clone() for t in sets[0]]
    one.run(*held)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = one.run(*held)
    # a second caller: the same weights, workspaces and stream of its own
    two = object.__new__(Layer)
    two.__dict__ = dict(one.__dict__, scratch=[torch.empty_like(s) for s in one.scratch])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for r in (1, 2, 3):
        for t, new in zip(held, sets[r]):
            t.copy_(new)
        g.replay()
        with torch.cuda.stream(side):
            want = two.run(*sets[r])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
