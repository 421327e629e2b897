"""Refusals of the F16 variant and of the layer's variants (no GPU, no kernel launched)."""

import pytest

import block_wise_int8_amd as bi8
from test_abi_fp8_cpu import ALIGN, CALLS, NULL, OK, SHAPE

F16 = bi8.GEMM_TILE_256X128_F16


def call(name, variant, **kw):
    a = {**CALLS[name], **kw}
    return getattr(bi8.load(), "blockint8_%s_variant" % name)(variant, *a.values(), None)


@pytest.mark.parametrize("name,variant,kw,status", [
    ("gemm_fp8", F16, dict(M=0), OK), ("gemm_fp8", F16, dict(K=250), ALIGN), ("gemm_fp8", F16, dict(xq=None), NULL),
    ("gemm_fp8", 7, {}, SHAPE), ("gemm_fp8", 9, {}, SHAPE), ("moe_gemm_fp8", F16, dict(R=0), OK),
    ("moe_gemm_fp8", F16, dict(K=200), ALIGN), ("moe_gemm_fp8", 9, {}, SHAPE),
    ("moe_layer_fp8", F16, dict(T=0), OK), ("moe_layer_fp8", F16, dict(x=None), NULL),
    ("moe_layer_fp8", F16, dict(nbytes=100), SHAPE), ("moe_layer_fp8", F16, dict(H=250, ldx=256), ALIGN)] + [
    ("moe_layer_fp8", v, {}, SHAPE) for v in (-1, 1, 2, 3, 4, 5, 6, 7, 9)])
def test_rules(name, variant, kw, status):
    assert call(name, variant, **kw) == status


def test_the_int8_products_do_not_have_it():
    P = 0x10000
    assert bi8.load().blockint8_gemm_variant(F16, P, P, P, P, None, P, 4, 256, 256, 128, 128, None) == SHAPE


def test_layer_select():
    for bad in ((0, 256, 256, 8, 2), (4, 250, 256, 8, 2), (4, 256, 256, 8, 9), (1 << 31, 256, 256, 8, 2)):
        assert bi8.moe_layer_fp8_select(*bad) == 0
    # a token, a batch and a prompt of a layer with large weights; a small layer
    assert bi8.moe_layer_fp8_select(1, 4096, 14336, 8, 2) == bi8.GEMM_SKINNY
    assert bi8.moe_layer_fp8_select(256, 4096, 14336, 8, 2) == F16
    assert bi8.moe_layer_fp8_select(4096, 4096, 14336, 8, 2) == bi8.GEMM_TILE_256X256
    assert bi8.moe_layer_fp8_select(300, 512, 384, 4, 2) == bi8.GEMM_TILE_128X64
