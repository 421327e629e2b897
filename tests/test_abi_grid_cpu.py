"""Sizes whose grid would hold 2^32 threads are refused before anything is launched (the runtime would report no
error and run the grid modulo 2^32).  No GPU: the pointers are never dereferenced."""

import pytest

import block_wise_int8_amd as bi8

P, HIP = 0x10000, 5

SKINNY, T128X64, T256X128, T256X256, T128X128 = 1, 2, 3, 4, 5


def dense(name, variant, M, N, K):
    lib = bi8.load()
    if name == "gemm_variant":
        return lib.blockint8_gemm_variant(variant, P, P, P, P, None, P, M, N, K, 128, 128, None)
    return lib.blockint8_gemm_fp8_variant(variant, P, P, P, P, None, P, M, N, K, 128, 128, None, 0, None)


def grouped(variant, R, N, K, E):
    return bi8.load().blockint8_moe_gemm_fp8_variant(variant, P, P, P, P, P, P, R, N, K, E, 128, 128, None, 0, None)


CALLS = {
    "fp8 streaming, 128 rows a workgroup": lambda: dense("fp8", SKINNY, 1, 1 << 30, 512),
    "fp8 streaming, 16 rows a workgroup": lambda: dense("fp8", SKINNY, 1, 1 << 27, 4096),
    "fp8 128 x 64": lambda: dense("fp8", T128X64, 1, 1 << 30, 16),
    "fp8 128 x 64, many rows": lambda: dense("fp8", T128X64, 1 << 29, 16, 16),
    "fp8 128 x 128": lambda: dense("fp8", T128X128, 1 << 16, 1 << 21, 16),
    "fp8 256 x 128": lambda: dense("fp8", T256X128, 1, (1 << 31) - 1, 16),
    "fp8 256 x 256": lambda: dense("fp8", T256X256, (1 << 31) - 1, 1, 16),
    "fp8 rows at any byte": lambda: dense("fp8", 0, 100, 1 << 30, 17),
    "fp8 grouped, streaming": lambda: grouped(SKINNY, 64, 1 << 24, 16, 64),
    "fp8 grouped, 128 x 64": lambda: grouped(T128X64, 64, 1 << 24, 16, 64),
    "fp8 grouped, 256 x 256": lambda: grouped(T256X256, 256, 1 << 23, 16, 65536),
    "fp8 gated": lambda: bi8.load().blockint8_moe_gemm_silu_quant_fp8(P, P, P, P, P, P, P, 64, 1 << 24, 16, 64, 128, 128,
                                                                      None),
    "int8 quantiser": lambda: bi8.load().blockint8_quant_act(P, 1 << 26, 8, 8, 128, P, P, None),
    "int8 quantiser, per token": lambda: bi8.load().blockint8_quant_act(P, 1 << 24, 8, 8, 8, P, P, None),
    "int8 gather": lambda: bi8.load().blockint8_quant_act_gather(P, 100, 8, P, 1 << 26, 8, 128, P, P, None),
    "int8 gating": lambda: bi8.load().blockint8_silu_mul_quant(P, 1 << 26, 16, 128, P, P, None, None),
    "int8 streaming": lambda: dense("gemm_variant", SKINNY, 1, 1 << 27, 16),
    "int8 128 x 64": lambda: dense("gemm_variant", T128X64, 1, 1 << 30, 16),
    "combine": lambda: bi8.load().blockint8_moe_combine(P, 1 << 20, P, P, 1 << 20, 1, 1 << 15, P, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused(name):
    assert CALLS[name]() == HIP
    assert b"invalid" in bi8.load().blockint8_last_error().lower()
