"""The router with scores, a bias and groups on the GPU against the oracle in binary64.

Whole numbers have to be equal.  Weights: the chosen scores, their sum and the scale are held in binary64 and rounded
once (2^-24), but for the softmax without a bias that is not renormalised, whose sum adds binary32 exponentials: with
x = max l - l each is off by x 2^-24 (its argument's rounding) and 2^-22 (two units of expf) of itself, and the mean of
x under the softmax is at most ln E <= 7, so the sum is within (7 + 4) 2^-24 of itself."""
import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import workloads as wl
from gpu_util import bf16_bits, bf16_to_dev, device, to_dev
from oracle import layer

pytestmark = pytest.mark.gpu


def logits_of(rng, T, E, bf16=False):
    l = (1.5 * rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)).astype(np.float32)
    if not bf16:
        return l, to_dev(l)
    bits = wl.to_bf16_bits(l)
    return layer.bf16(bits), bf16_to_dev(bits)


def check(out, logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renormalize=False, scale=1.0):
    ids, w, st, off, row_of = (t.cpu().numpy() for t in out)
    want, wt = layer.route_grouped(logits, k, score, bias, groups, topk_groups, group_top, renormalize, scale)
    assert np.array_equal(ids, want)
    units = 12 if score == "softmax" and bias is None and not renormalize else 1
    assert np.all(np.abs(w - wt) <= units * 1.01 * 2.0 ** -24 * np.abs(wt) + 2.0 ** -149)
    want_st, want_off, want_row = layer.dispatch(want, np.shape(logits)[1])
    assert np.array_equal(off, want_off) and np.array_equal(st, want_st) and np.array_equal(row_of, want_row)


SHAPES = [  # T, E, k, groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 2, 2, 2, 2, 1), (5, 3, 2, 3, 2, 2), (16, 8, 8, 1, 1, 1),
    (17, 8, 3, 4, 2, 2), (15, 64, 6, 1, 1, 1), (64, 128, 8, 1, 1, 1), (33, 160, 6, 8, 3, 1), (40, 160, 32, 8, 3, 2),
    (100, 60, 5, 20, 7, 2), (70, 256, 16, 64, 9, 2), (130, 384, 10, 3, 2, 2), (50, 512, 17, 4, 1, 1),
    (20, 1024, 32, 32, 20, 2), (35, 1023, 9, 33, 5, 2), (9, 1020, 9, 5, 3, 1), (12, 1000, 8, 1, 1, 1), (18, 1024, 4, 64, 64, 1),
    (1025, 16, 2, 1, 1, 1), (1100, 33, 4, 11, 5, 2), (2048, 256, 8, 8, 4, 2), (1500, 128, 8, 1, 1, 1), (1200, 500, 8, 4, 2, 2),
    (1030, 700, 8, 7, 3, 1), (4097, 40, 3, 8, 2, 2), (5000, 8, 2, 1, 1, 1), (8193, 16, 4, 16, 6, 1)]


@pytest.mark.parametrize("T,E,k,groups,topk_groups,group_top", SHAPES)
@pytest.mark.parametrize("score,bias,renormalize,scale,bf16", [
    ("softmax", False, False, 1.0, False), ("softmax", True, True, 2.5, True), ("sigmoid", True, True, 2.5, False),
    ("sigmoid", False, False, 16.0, True), ("softmax", False, True, 1.0, True)])
def test_against_oracle(T, E, k, groups, topk_groups, group_top, score, bias, renormalize, scale, bf16):
    rng = wl.rng_for((111, T, E))
    l, ld = logits_of(rng, T, E, bf16)
    b = (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None
    kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_top=group_top, renormalize=renormalize,
              scale=scale)
    out = bi8.moe_route_grouped(ld, k, bias=None if b is None else to_dev(b), **kw)
    check(out, l, k, bias=b, **kw)


@pytest.mark.parametrize("T", [20001, 40000])
def test_many_tokens(T):
    """Past what one workgroup's sums cover; the dispatch by numpy's stable sort."""
    rng = wl.rng_for((112, T))
    E, k = 24, 2
    l, ld = logits_of(rng, T, E)
    ids, w, st, off, row_of = (t.cpu().numpy() for t in bi8.moe_route_grouped(ld, k, renormalize=True))
    assert np.array_equal(ids, np.argsort(-l, axis=1, kind="stable")[:, :k])
    order = np.argsort(ids.ravel(), kind="stable")
    assert np.array_equal(st, order // k) and np.array_equal(off, np.searchsorted(ids.ravel()[order], np.arange(E + 1)))
    back = np.empty(T * k, np.int64)
    back[order] = np.arange(T * k)
    assert np.array_equal(row_of.ravel(), back)


@pytest.mark.parametrize("T", [7, 40, 1100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_masks(T, score):
    """Few distinct logits, experts and rows off, infinities and NaN, a bias that switches off."""
    rng = wl.rng_for((113, T))
    E, k = 48, 6
    l = rng.integers(-2, 3, (T, E)).astype(np.float32)
    l[:, ::5] = -np.inf
    l[rng.random((T, E)) < 0.05] = -0.0
    l[1] = -np.inf
    l[2, 3:] = np.nan
    l[3, [7, 30]] = np.inf
    l[4] = np.finfo(np.float32).min
    l[5] = -300.0
    l[5, 11] = -200.0
    for kw in (dict(), dict(groups=6, topk_groups=2, group_top=1), dict(groups=6, topk_groups=2, group_top=2),
               dict(renormalize=True, scale=2.0)):
        check(bi8.moe_route_grouped(to_dev(l), k, score=score, **kw), l, k, score=score, **kw)
        b = (0.25 * rng.integers(-1, 2, E)).astype(np.float32)   # ties of sums are ties in binary64 too
        b[3] = -np.inf
        b[9] = np.nan
        if kw.get("group_top") != 2:
            check(bi8.moe_route_grouped(to_dev(l), k, score=score, bias=to_dev(b), **kw), l, k, score=score, bias=b, **kw)


def test_lowest_value_of_bf16_as_a_mask():
    rng = wl.rng_for(114)
    bits = wl.to_bf16_bits(rng.standard_normal((30, 32)).astype(np.float32))
    bits[rng.random((30, 32)) < 0.6] = 0xFF7F
    bits[4] = 0xFF7F
    check(bi8.moe_route_grouped(bf16_to_dev(bits), 4), layer.bf16(bits), 4)
    check(bi8.moe_route_grouped(bf16_to_dev(bits), 4, score="sigmoid", renormalize=True), layer.bf16(bits), 4,
          score="sigmoid", renormalize=True)


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_apart_and_given_outputs(bf16):
    rng = wl.rng_for(115)
    T, E, k = 50, 40, 3
    l, ld = logits_of(rng, T, E + 7, bf16)
    n = bi8.moe_route_grouped_workspace_size(T, E)
    dev = device()
    out = tuple(torch.full(s, -9, dtype=d, device=dev) for s, d in (((T, k), torch.int32), ((T, k), torch.float32),
                                                                 ((T * k,), torch.int32), ((E + 1,), torch.int32),
                                                                 ((T, k), torch.int32)))
    scratch = torch.full((n + 64,), 0xAB, dtype=torch.uint8, device=dev)
    got = bi8.moe_route_grouped(ld[:, 3: 3 + E], k, out=out, workspace=scratch[:n], renormalize=True)
    assert all(a is b for a, b in zip(got, out))
    check(got, l[:, 3: 3 + E], k, renormalize=True)
    assert torch.all(scratch[n:] == 0xAB)


def test_no_tokens():
    out = bi8.moe_route_grouped(torch.empty(0, 12, device=device()), 2, groups=3, topk_groups=2)
    assert out[0].shape == (0, 2) and out[3].tolist() == [0] * 13


def test_refusals_of_the_binding():
    l = torch.zeros(4, 8, device=device())
    for bad in (lambda: bi8.moe_route_grouped(l.double(), 2), lambda: bi8.moe_route_grouped(l.half(), 2),
                lambda: bi8.moe_route_grouped(l[0], 2), lambda: bi8.moe_route_grouped(l, 2, bias=l[0].double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bi8.moe_route_grouped(l, 2, score="tanh"), lambda: bi8.moe_route_grouped(l, 2, bias=l[0, :7]),
                lambda: bi8.moe_route_grouped(l.t(), 2), lambda: bi8.moe_route_grouped(l, 2, bias=l[0].cpu()),
                lambda: bi8.moe_route_grouped(l, 2, out=bi8.moe_route_grouped(l, 3))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bi8.moe_route_grouped(l, 9), lambda: bi8.moe_route_grouped(l, 2, groups=3),
                lambda: bi8.moe_route_grouped(l, 3, groups=4, topk_groups=1)):
        with pytest.raises(bi8.BlockInt8Error):
            bad()


@pytest.mark.parametrize("T", [5, 300])
def test_captured_and_replayed(T):
    rng = wl.rng_for((116, T))
    E, k = 64, 8
    ls = [logits_of(rng, T, E)[1] for _ in range(4)]
    bias = to_dev((0.1 * rng.standard_normal(E)).astype(np.float32))
    kw = dict(score="sigmoid", bias=bias, groups=8, topk_groups=4, group_top=2, renormalize=True)
    l, dev = ls[0].clone(), device()
    out = bi8.moe_route_grouped(l, k, **kw)
    scratch = torch.empty(max(16, bi8.moe_route_grouped_workspace_size(T, E)), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bi8.moe_route_grouped(l, k, out=out, workspace=scratch, **kw)
    for r in (1, 2, 3):
        l.copy_(ls[r])
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, bi8.moe_route_grouped(ls[r], k, **kw)):
            assert torch.equal(a, b)


# ------------------------------------------------------------ the MoE layers --

def fp8_weights(rng, E, N, K):
    w = [bi8.quant_weight_fp8(bf16_to_dev(wl.activations(rng, N, K))) for _ in range(E)]
    return torch.stack([q.view(torch.uint8) for q, _ in w]).view(torch.float8_e4m3fn), torch.stack([s for _, s in w])


@pytest.mark.parametrize("T,I", [(1, 128), (9, 256), (70, 96), (300, 128)])
def test_layers_take_the_routing(T, I):
    """The same routing by moe_route gives the layers the same bits as their logits do."""
    rng = wl.rng_for((117, T))
    H, E, k = 256, 12, 3
    x, logits = bf16_to_dev(wl.activations(rng, T, H)), to_dev(wl.router_logits(rng, T, E))
    w13, ws13 = fp8_weights(rng, E, 2 * I, H)
    w2, ws2 = fp8_weights(rng, E, H, I)
    route = bi8.moe_route(logits, k)
    a = bi8.moe_layer_fp8(x, logits, w13, ws13, w2, ws2, k)
    assert torch.equal(a, bi8.moe_layer_fp8(x, None, w13, ws13, w2, ws2, k, route=route))
    b13, b2 = (to_dev(wl.weights(rng, E, 2 * I, H)), to_dev(wl.weights(rng, E, H, I)))
    a = bi8.moe_layer(x, logits, b13, ws13, b2, ws2, k)
    assert torch.equal(a, bi8.moe_layer(x, None, b13, ws13, b2, ws2, k, route=route))
    for bad in (lambda: bi8.moe_layer_fp8(x, logits, w13, ws13, w2, ws2, k, route=route),
                lambda: bi8.moe_layer_fp8(x, None, w13, ws13, w2, ws2, k + 1, route=route),
                lambda: bi8.moe_layer_fp8(x, None, w13, ws13, w2, ws2, k, True, route=route),
                lambda: bi8.moe_layer(x, logits, b13, ws13, b2, ws2, k, route=route),
                lambda: bi8.moe_layer(x, None, b13, ws13, b2, ws2, 2, route=route)):
        with pytest.raises(ValueError):
            bad()


def test_layer_of_more_experts_than_eight_a_token():
    """k = 12 of 16 experts: the layer against its steps, one call each."""
    rng = wl.rng_for(118)
    T, H, I, E, k = 21, 128, 128, 16, 12
    x = bf16_to_dev(wl.activations(rng, T, H))
    l, ld = logits_of(rng, T, E, True)
    w13, ws13 = fp8_weights(rng, E, 2 * I, H)
    w2, ws2 = fp8_weights(rng, E, H, I)
    route = bi8.moe_route_grouped(ld, k, "sigmoid", groups=4, topk_groups=3, renormalize=True)
    _, w, st, off, row_of = route
    out = bi8.moe_layer_fp8(x, None, w13, ws13, w2, ws2, k, route=route)
    h = bi8.moe_gemm_fp8(*bi8.quant_act_gather_fp8(x, st), off, w13, ws13,
                         variant=bi8.moe_layer_fp8_select(T * 3, H, I, E, 4) or None)
    y = bi8.moe_gemm_fp8(*bi8.silu_mul_quant_fp8(h), off, w2, ws2)
    ref = bi8.moe_combine(y, row_of, w)
    d, r = (out.double() - ref.double()).cpu(), ref.double().cpu()
    # sums in another order: a code of the second quantiser may move by a step (2^-4 of some values)
    assert d.norm() <= 2.0 ** -6 * r.norm() and bf16_bits(out).any()
