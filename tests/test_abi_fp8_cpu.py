"""Host-side checks of the e4m3 and norm entry points (no GPU, no kernel launched): every declared
function is exported, and every bad argument is refused with the documented status before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

import block_wise_int8_amd as bi8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, BLOCK, ALIGN = 0, 1, 2, 3, 4
P = 0x10000          # a fake, 16-byte aligned address (never dereferenced)
ODD = 0x10001

# name -> default arguments that only the pointers' being fake makes invalid to run
CALLS = {
    "quant_act_fp8": dict(x=P, M=4, K=200, ldx=200, bk=128, xq=P, xs=P),
    "quant_act_gather_fp8": dict(x=P, T=4, ldx=200, rows=P, R=4, K=200, bk=128, xq=P, xs=P),
    "silu_mul_quant_fp8": dict(h=P, R=4, I=256, bk=128, aq=P, as_=P, a=None),
    "quant_weight_fp8": dict(w=P, N=4, K=200, ldw=200, bn=128, bk=128, wq=P, ws=P),
    "gemm_fp8": dict(xq=P, xs=P, w=P, ws=P, bias=None, y=P, M=4, N=256, K=256, bn=128, bk=128, wsp=None, nbytes=0),
    "linear_fp8": dict(x=P, ldx=256, w=P, ws=P, bias=None, y=P, M=4, N=256, K=256, bn=128, bk=128, xq=P, xs=P,
                       wsp=None, nbytes=0),
    "moe_gemm_fp8": dict(xq=P, xs=P, off=P, w=P, ws=P, y=P, R=4, N=256, K=256, E=2, bn=128, bk=128, wsp=None,
                         nbytes=0),
    "moe_gemm_silu_quant_fp8": dict(xq=P, xs=P, off=P, w13=P, ws13=P, aq=P, as_=P, R=4, I=256, K=256, E=2, bn=128,
                                    bk=128),
    "moe_layer_fp8": dict(x=P, ldx=256, logits=P, w13=P, ws13=P, w2=P, ws2=P, out=P, T=4, H=256, I=256, E=8, k=2, renorm=0,
                          bn=128, bk=128, wsp=P, nbytes=1 << 30),
    "rmsnorm_quant": dict(x=P, ldx=256, residual=P, ldr=256, weight=P, eps=1e-6, M=4, H=256, bk=128, h=P, ldh=256,
                          y=None, xq=P, xs=P),
}
CALLS["rmsnorm_quant_fp8"] = CALLS["rmsnorm_quant"]

NORM_BAD = [
    (dict(x=None), NULL), (dict(weight=None), NULL), (dict(xq=None), NULL), (dict(xs=None), NULL),
    (dict(h=None), NULL), (dict(residual=None), NULL),   # h belongs to a residual, and a residual needs it
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(H=0), SHAPE), (dict(H=1 << 24), SHAPE),
    (dict(ldx=255), SHAPE), (dict(ldr=255), SHAPE), (dict(ldh=255), SHAPE),
    (dict(eps=-1e-9), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(bk=256), BLOCK), (dict(bk=0), BLOCK),
    (dict(x=ODD), ALIGN), (dict(residual=ODD), ALIGN), (dict(weight=ODD), ALIGN), (dict(h=ODD), ALIGN),
    (dict(y=ODD), ALIGN), (dict(xq=P + 8), ALIGN), (dict(xs=P + 2), ALIGN),
]
PRODUCT_BAD = [
    (dict(xq=None), NULL), (dict(xs=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL),
    (dict(N=0), SHAPE), (dict(N=1 << 31), SHAPE), (dict(K=0), SHAPE), (dict(K=1 << 24, ldx=1 << 24), SHAPE),
    (dict(nbytes=-1), SHAPE), (dict(bn=64), BLOCK), (dict(bk=0), BLOCK), (dict(bn=1, bk=256), BLOCK),
    (dict(xq=P + 4), ALIGN), (dict(w=P + 8), ALIGN), (dict(xs=P + 1), ALIGN), (dict(ws=P + 2), ALIGN),
    (dict(y=ODD), ALIGN), (dict(wsp=P + 8, nbytes=1 << 30), ALIGN),
]
BAD = {
    "quant_act_fp8": [
        (dict(x=None), NULL), (dict(xq=None), NULL), (dict(xs=None), NULL), (dict(M=-1), SHAPE), (dict(K=0), SHAPE),
        (dict(K=1 << 24, ldx=1 << 24), SHAPE), (dict(ldx=199), SHAPE), (dict(bk=200), BLOCK), (dict(bk=-1), BLOCK),
        (dict(x=ODD), ALIGN), (dict(xq=P + 8), ALIGN), (dict(xs=P + 2), ALIGN)],
    "quant_act_gather_fp8": [
        (dict(x=None), NULL), (dict(rows=None), NULL), (dict(xq=None), NULL), (dict(R=-1), SHAPE), (dict(T=-1), SHAPE),
        (dict(ldx=10), SHAPE), (dict(bk=64), BLOCK), (dict(rows=P + 2), ALIGN), (dict(x=ODD), ALIGN)],
    "silu_mul_quant_fp8": [
        (dict(h=None), NULL), (dict(aq=None), NULL), (dict(as_=None), NULL), (dict(R=-1), SHAPE), (dict(I=0), SHAPE),
        (dict(I=250), ALIGN), (dict(bk=256), BLOCK), (dict(h=P + 8), ALIGN), (dict(a=P + 2), ALIGN)],
    "quant_weight_fp8": [
        (dict(w=None), NULL), (dict(wq=None), NULL), (dict(ws=None), NULL), (dict(N=-1), SHAPE),
        (dict(N=65535 * 128 + 1), SHAPE), (dict(K=0), SHAPE), (dict(ldw=199), SHAPE), (dict(bn=64), BLOCK),
        (dict(w=ODD), ALIGN), (dict(wq=P + 4), ALIGN), (dict(ws=P + 2), ALIGN)],
    "gemm_fp8": [b for b in PRODUCT_BAD if "ldx" not in b[0]] + [
        (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=1 << 24), SHAPE), (dict(bias=ODD), ALIGN)],
    "linear_fp8": PRODUCT_BAD + [
        (dict(x=None), NULL), (dict(M=-1), SHAPE), (dict(ldx=255), SHAPE), (dict(x=ODD), ALIGN),
        (dict(bias=ODD), ALIGN)],
    "moe_gemm_fp8": [b for b in PRODUCT_BAD if "ldx" not in b[0]] + [
        (dict(off=None), NULL), (dict(off=P + 2), ALIGN), (dict(E=0), SHAPE), (dict(E=65537), SHAPE),
        (dict(R=-1), SHAPE), (dict(K=100), ALIGN)],
    "moe_gemm_silu_quant_fp8": [
        (dict(xq=None), NULL), (dict(xs=None), NULL), (dict(off=None), NULL), (dict(w13=None), NULL),
        (dict(ws13=None), NULL), (dict(aq=None), NULL), (dict(as_=None), NULL), (dict(R=-1), SHAPE),
        (dict(R=1 << 31), SHAPE), (dict(I=0), SHAPE), (dict(I=200), SHAPE), (dict(I=1 << 30), SHAPE),
        (dict(K=0), SHAPE), (dict(K=100), ALIGN), (dict(E=0), SHAPE), (dict(E=65537), SHAPE), (dict(bn=64), BLOCK),
        (dict(bk=64), BLOCK), (dict(off=P + 2), ALIGN), (dict(xq=P + 8), ALIGN), (dict(xs=P + 2), ALIGN),
        (dict(w13=P + 8), ALIGN), (dict(ws13=P + 2), ALIGN), (dict(aq=P + 8), ALIGN), (dict(as_=P + 2), ALIGN)],
    "moe_layer_fp8": [(dict([(name, None)]), NULL) for name in ("x", "logits", "w13", "ws13", "w2", "ws2", "out", "wsp")] + [
        (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE), (dict(H=0), SHAPE), (dict(I=0), SHAPE), (dict(E=0), SHAPE),
        (dict(H=1 << 24, ldx=1 << 24), SHAPE), (dict(I=1 << 24), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE),
        (dict(k=9), SHAPE), (dict(E=1), SHAPE), (dict(ldx=255), SHAPE), (dict(nbytes=0), SHAPE), (dict(nbytes=-1), SHAPE),
        (dict(nbytes=4096), SHAPE), (dict(H=248), ALIGN), (dict(I=40), ALIGN), (dict(bn=64), BLOCK), (dict(bk=1), BLOCK),
        (dict(x=ODD), ALIGN), (dict(logits=P + 2), ALIGN), (dict(w13=P + 8), ALIGN), (dict(ws13=P + 2), ALIGN),
        (dict(w2=P + 8), ALIGN), (dict(ws2=P + 2), ALIGN), (dict(out=P + 8), ALIGN), (dict(wsp=P + 128), ALIGN)],
    "rmsnorm_quant": NORM_BAD, "rmsnorm_quant_fp8": NORM_BAD,
}


def run(name, **kw):
    args = dict(CALLS[name], **kw)
    assert list(args) == list(CALLS[name]), "unknown argument"
    return getattr(bi8.load(), "blockint8_" + name)(*args.values(), None)


@pytest.mark.parametrize("name,kw,status", [(n, kw, st) for n, cases in BAD.items() for kw, st in cases])
def test_refusals(name, kw, status):
    assert run(name, **kw) == status
    assert bi8.load().blockint8_last_error().decode().startswith("blockint8_" + name + ":")


@pytest.mark.parametrize("name", sorted(CALLS))
def test_empty_is_a_no_op(name):
    size = next(k for k in ("M", "R", "N", "T") if k in CALLS[name])
    none = {k: None for k, v in CALLS[name].items() if v == P}
    assert run(name, **{**none, size: 0}) == OK
    assert bi8.load().blockint8_last_error().decode() == ""


@pytest.mark.parametrize("header", ["blockint8_fp8.h", "blockint8_norm.h"])
def test_every_declared_function_is_exported(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(blockint8_\w+)\s*\(", text))
    assert names
    raw = ctypes.CDLL(bi8.lib_path())
    for name in names:
        getattr(raw, name)
    wanted = {"blockint8_" + n for n in CALLS if ("norm" in n) == ("norm" in header)}
    assert wanted <= names


def test_variant_rules():
    lib, a = bi8.load(), list(CALLS["gemm_fp8"].values())
    assert lib.blockint8_gemm_fp8_variant(6, *a, None) == SHAPE
    assert lib.blockint8_gemm_fp8_variant(-1, *a, None) == SHAPE
    a[list(CALLS["gemm_fp8"]).index("K")] = 250
    assert lib.blockint8_gemm_fp8_variant(3, *a, None) == ALIGN
    assert lib.blockint8_moe_gemm_fp8_variant(6, *CALLS["moe_gemm_fp8"].values(), None) == SHAPE
    for M, N, K in [(1, 4096, 4096), (64, 8192, 4096), (333, 5000, 4000), (4096, 4096, 4096), (2048, 28672, 4096)]:
        assert 1 <= bi8.gemm_fp8_select(M, N, K) <= 5 and 1 <= bi8.moe_gemm_fp8_select(M, N, K, 8) <= 5


def test_workspace_sizes_of_bad_problems_are_zero():
    assert bi8.gemm_fp8_workspace_size(0, 10, 10) == 0 and bi8.gemm_fp8_workspace_size(10, -1, 10) == 0
    for bad in ((0, 256, 256, 8, 2), (4, 250, 256, 8, 2), (4, 256, 24, 8, 2), (4, 256, 256, 8, 9), (4, 256, 256, 0, 1),
                (1 << 31, 256, 256, 8, 2), (4, 256, 0, 8, 2), (4, 256, 256, 2, 3)):
        assert bi8.moe_layer_fp8_workspace_size(*bad) == 0
    assert bi8.moe_layer_fp8_workspace_size(4, 256, 256, 8, 2) > 4 * 2 * 256 * 4
    assert bi8.moe_gemm_fp8_workspace_size(8, 10, 100, 2) == 0 and bi8.moe_gemm_fp8_workspace_size(8, 10, 128, 0) == 0


def test_binding_has_no_cpu_path():
    f8 = torch.float8_e4m3fn
    x, xq = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=f8)
    s, w, ws = torch.zeros(4, 1), torch.zeros(8, 128, dtype=f8), torch.zeros(1, 1)
    off = torch.zeros(2, dtype=torch.int32)
    for fn in (lambda: bi8.quant_act_fp8(x), lambda: bi8.quant_act_gather_fp8(x, off),
               lambda: bi8.silu_mul_quant_fp8(x), lambda: bi8.quant_weight_fp8(x), lambda: bi8.gemm_fp8(xq, s, w, ws),
               lambda: bi8.linear_fp8(x, w, ws), lambda: bi8.moe_gemm_fp8(xq, s, off, w[None], ws[None]),
               lambda: bi8.moe_gemm_silu_quant_fp8(xq, s, off, w[None], ws[None]),
               lambda: bi8.moe_layer_fp8(x, s, w[None], ws[None], w[None], ws[None], 1),
               lambda: bi8.rmsnorm_quant(x, x[0])):
        with pytest.raises(ValueError, match="HIP device"):
            fn()
