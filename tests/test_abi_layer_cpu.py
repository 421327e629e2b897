"""Host-side checks of the operators beside the 8-bit products (no GPU, no kernel launched): every declared function
is exported, and every bad argument is refused with the documented status before any HIP call."""
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


def sections(*n):
    return (ctypes.c_int32 * len(n))(*n)


def widths(*n):
    return (ctypes.c_int64 * len(n))(*n)


# name -> default arguments that only the pointers' being fake makes invalid to run
CALLS = {
    "qk_norm_rope": dict(q=P, q_token=384, q_head=64, Hq=4, k=P, k_token=384, k_head=64, Hk=2, q_weight=P, k_weight=P,
                         eps=1e-6, table=P, P=16, positions=P, positions_axis=0, axes=1, sections=sections(32),
                         interleaved=0, T=3, D=64, rot=64, q_out=P, qo_token=256, qo_head=64, k_out=P, ko_token=128,
                         ko_head=64),
    "lora_add": dict(x=P, ldx=64, a=P, b=P, scales=P, adapter=P, y=P, ldy=96, M=5, N=96, K=64, L=3, R=16, parts=2,
                     widths=widths(64, 32), wsp=P, nbytes=1 << 20),
    "moe_route_grouped": dict(logits=P, bf16=0, ldl=64, bias=P, T=100, E=64, k=4, score=1, groups=8, topk_groups=2,
                              group_top=2, renorm=1, scale=1.0, ids=P, weights=P, st=P, off=P, row_of=P, wsp=P,
                              nbytes=1 << 20),
    "moe_layer_fp8_routed": dict(variant=0, x=P, ldx=256, weights=P, st=P, off=P, row_of=P, w13=P, ws13=P, w2=P, ws2=P,
                                 out=P, T=4, H=256, I=256, E=16, k=9, bn=128, bk=128, wsp=P, nbytes=1 << 30),
}

BAD = {
    "qk_norm_rope": [
        (dict(q=None), NULL), (dict(k=None), NULL), (dict(table=None), NULL), (dict(positions=None), NULL),
        (dict(q_out=None), NULL), (dict(k_out=None), NULL), (dict(sections=None), NULL),
        (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(Hq=0), SHAPE), (dict(Hk=-1), SHAPE), (dict(Hq=1 << 17), SHAPE),
        (dict(D=63), SHAPE), (dict(D=0), SHAPE), (dict(D=1026), SHAPE), (dict(rot=0), SHAPE), (dict(rot=63), SHAPE),
        (dict(rot=66), SHAPE), (dict(P=0), SHAPE), (dict(P=1 << 31), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5), SHAPE),
        (dict(positions_axis=-1), SHAPE), (dict(sections=sections(31)), SHAPE), (dict(sections=sections(33)), SHAPE),
        (dict(axes=2, sections=sections(-1, 33)), SHAPE), (dict(axes=2, sections=sections(32, 32)), SHAPE),
        (dict(eps=-1e-9), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
        (dict(q_token=-1), SHAPE), (dict(k_head=-64), SHAPE), (dict(q_token=1 << 41), SHAPE),
        # outputs whose heads share elements: apart by less than a head, tokens inside each other's heads
        (dict(qo_head=63), SHAPE), (dict(qo_token=255), SHAPE), (dict(qo_token=0), SHAPE), (dict(ko_head=0), SHAPE),
        (dict(qo_token=64, qo_head=191), SHAPE), (dict(qo_token=64, qo_head=128), SHAPE),
        (dict(q=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(q_weight=ODD), ALIGN), (dict(k_weight=ODD), ALIGN),
        (dict(table=P + 2), ALIGN), (dict(positions=P + 2), ALIGN), (dict(q_out=ODD), ALIGN), (dict(k_out=ODD), ALIGN)],
    "lora_add": [(dict([(name, None)]), NULL) for name in ("x", "a", "b", "adapter", "y", "widths", "wsp")] + [
        (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=0), SHAPE), (dict(N=1 << 31), SHAPE), (dict(K=0), SHAPE),
        (dict(K=1 << 24, ldx=1 << 24), SHAPE), (dict(ldx=(1 << 23) + 1), SHAPE), (dict(ldy=(1 << 23) + 1), SHAPE),
        (dict(N=(1 << 23) + 1, ldy=1 << 25, widths=widths(1 << 23, 1)), SHAPE), (dict(L=0), SHAPE), (dict(L=(1 << 24) + 1), SHAPE), (dict(R=0), SHAPE),
        (dict(R=136), SHAPE), (dict(R=-8), SHAPE), (dict(parts=0), SHAPE), (dict(parts=5), SHAPE),
        (dict(widths=widths(64, 31)), SHAPE), (dict(widths=widths(96, 0)), SHAPE), (dict(widths=widths(97, -1)), SHAPE),
        (dict(ldx=63), SHAPE), (dict(ldy=95), SHAPE), (dict(nbytes=5 * 32 * 4 - 1), SHAPE), (dict(nbytes=-1), SHAPE),
        (dict(R=12), ALIGN), (dict(x=ODD), ALIGN), (dict(a=P + 8), ALIGN), (dict(b=P + 2), ALIGN),
        (dict(scales=P + 2), ALIGN), (dict(adapter=P + 1), ALIGN), (dict(y=ODD), ALIGN), (dict(wsp=P + 8), ALIGN)],
    "moe_route_grouped": [(dict([(name, None)]), NULL) for name in ("logits", "ids", "weights", "st", "off", "row_of")] + [
        (dict(T=-1), SHAPE), (dict(T=1 << 29), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE),
        (dict(k=33), SHAPE), (dict(E=8, k=9), SHAPE), (dict(ldl=63), SHAPE), (dict(score=2), SHAPE), (dict(score=-1), SHAPE),
        (dict(groups=0), SHAPE), (dict(groups=7), SHAPE), (dict(groups=128, E=128), SHAPE), (dict(topk_groups=0), SHAPE),
        (dict(topk_groups=9), SHAPE), (dict(k=17), SHAPE), (dict(groups=64, topk_groups=3), SHAPE), (dict(group_top=0), SHAPE),
        (dict(group_top=3), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
        (dict(wsp=None), SHAPE), (dict(nbytes=7 * 64 - 1), SHAPE), (dict(nbytes=-1), SHAPE), (dict(logits=P + 2), ALIGN),
        (dict(logits=ODD, bf16=1), ALIGN), (dict(bias=P + 2), ALIGN), (dict(ids=P + 2), ALIGN), (dict(weights=P + 1), ALIGN),
        (dict(st=P + 2), ALIGN), (dict(off=P + 2), ALIGN), (dict(row_of=P + 2), ALIGN), (dict(wsp=P + 8), ALIGN)],
    "moe_layer_fp8_routed": [(dict([(name, None)]), NULL) for name in ("x", "weights", "st", "off", "row_of", "w13", "ws13",
                                                                     "w2", "ws2", "out", "wsp")] + [
        (dict(variant=1), SHAPE), (dict(variant=-1), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE), (dict(H=0), SHAPE),
        (dict(I=0), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=17), SHAPE),
        (dict(E=64, k=33), SHAPE), (dict(ldx=255), SHAPE), (dict(nbytes=0), SHAPE), (dict(nbytes=4096), SHAPE), (dict(H=248), ALIGN),
        (dict(I=40), ALIGN), (dict(bn=64), BLOCK), (dict(bk=1), BLOCK), (dict(x=ODD), ALIGN), (dict(weights=P + 2), ALIGN),
        (dict(st=P + 2), ALIGN), (dict(off=P + 2), ALIGN), (dict(row_of=P + 2), ALIGN), (dict(w13=P + 8), ALIGN),
        (dict(ws13=P + 2), ALIGN), (dict(w2=P + 8), ALIGN), (dict(ws2=P + 2), ALIGN), (dict(out=P + 8), ALIGN),
        (dict(wsp=P + 128), ALIGN)],
}
# calls that write something even without tokens
NOT_EMPTY = {"moe_route_grouped"}


def run(name, **kw):
    args = dict(CALLS[name], **kw)
    assert list(args) == list(CALLS[name]), "unknown argument"
    return getattr(bi8.load(), "blockint8_" + name)(*args.values(), None)


@pytest.mark.parametrize("name,kw,status", [(n, kw, st) for n, cases in BAD.items() for kw, st in cases])
def test_refusals(name, kw, status):
    assert run(name, **kw) == status
    assert bi8.load().blockint8_last_error().decode().startswith("blockint8_" + name + ":")


@pytest.mark.parametrize("name", sorted(set(CALLS) - NOT_EMPTY))
def test_empty_is_a_no_op(name):
    size = next(k for k in ("M", "R", "N", "T") if k in CALLS[name])
    none = {k: None for k, v in CALLS[name].items() if v == P}
    assert run(name, **{**none, size: 0}) == OK
    assert bi8.load().blockint8_last_error().decode() == ""


@pytest.mark.parametrize("header", ["blockint8_heads.h", "blockint8_route.h", "blockint8_lora.h"])
def test_every_declared_function_is_exported(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(blockint8_\w+)\s*\(", text))
    assert names
    raw = ctypes.CDLL(bi8.lib_path())
    for name in names:
        getattr(raw, name)


def test_binding_has_no_cpu_path():
    x = torch.zeros(4, 2, 8, dtype=torch.bfloat16)
    for fn in (lambda: bi8.qk_norm_rope(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8)),
               lambda: bi8.moe_route_grouped(torch.zeros(4, 8), 2),
               lambda: bi8.lora_add(x[0], x[0], x, x, torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="HIP device"):
            fn()


def test_workspace_sizes():
    size = bi8.moe_route_grouped_workspace_size
    assert size(0, 64) == size(-1, 64) == size(100, 0) == size(100, 1025) == size(1 << 31, 64) == size(16, 64) == 0
    assert size(17, 64) > 0 and size(100, 64) == 7 * 64 and size(1 << 20, 1024) > (1 << 14) * 1024 * 5
    routed = bi8.moe_layer_fp8_workspace_size(4, 256, 256, 16, 9, routed=True)
    assert routed > 0 and bi8.moe_layer_fp8_workspace_size(4, 256, 256, 16, 9) == 0
    assert bi8.moe_layer_fp8_workspace_size(4, 256, 256, 16, 33, routed=True) == 0
    assert bi8.moe_layer_fp8_workspace_size(4, 256, 256, 16, 2, True) < bi8.moe_layer_fp8_workspace_size(4, 256, 256, 16, 2)
    size = bi8.lora_add_workspace_size
    assert size(0, 64, 8) == size(-1, 64, 8) == size(5, 0, 8) == size(5, 64, 12) == size(5, 64, 264) == 0
    assert size(5, 64, 136, 2) == size(5, 64, 8, 0) == size(5, 64, 8, 5) == size(1 << 31, 64, 8) == 0
    assert size(5, 64, 16, 2) == 5 * 32 * 4 and size(1, 4096, 16) % (16 * 4) == 0


def test_grids_of_too_many_threads_are_refused():
    """Before either launch (the runtime would report no error and run the grid modulo 2^32)."""
    lib, P, HIP = bi8.load(), 0x10000, 5
    for M, L, parts in ((1 << 29, 1, (1,)),        # the first product's grid
                        (1 << 28, 1, (1,) * 4),    # the second's: a workgroup at least for each part
                        (1 << 27, 100, (4,))):
        n = lib.blockint8_lora_add_workspace_size(M, 1, 8, len(parts))
        status = lib.blockint8_lora_add(P, 1, P, P, None, P, P, sum(parts), M, sum(parts), 1, L, 8, len(parts),
                                        (ctypes.c_int64 * len(parts))(*parts), P, n, None)
        assert (status, b"invalid" in lib.blockint8_last_error().lower()) == (HIP, True), (M, L, parts)
