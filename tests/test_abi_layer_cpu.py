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


# name -> default arguments that only the pointers' being fake makes invalid to run
CALLS = {
    "qk_norm_rope": dict(q=P, q_token=384, q_head=64, Hq=4, k=P, k_token=384, k_head=64, Hk=2, q_weight=P, k_weight=P,
                         eps=1e-6, table=P, P=16, positions=P, positions_axis=0, axes=1, sections=sections(32),
                         interleaved=0, T=3, D=64, rot=64, q_out=P, qo_token=256, qo_head=64, k_out=P, ko_token=128,
                         ko_head=64),
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


@pytest.mark.parametrize("header", ["blockint8_heads.h"])
def test_every_declared_function_is_exported(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(blockint8_\w+)\s*\(", text))
    assert names
    raw = ctypes.CDLL(bi8.lib_path())
    for name in names:
        getattr(raw, name)


def test_binding_has_no_cpu_path():
    x = torch.zeros(4, 2, 8, dtype=torch.bfloat16)
    for fn in (lambda: bi8.qk_norm_rope(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8)),):
        with pytest.raises(ValueError, match="HIP device"):
            fn()
