"""The library's own machine code: what a wide store writes is left alone while the store reads it.

A store of three or four registers reads them after it was issued.  A vector instruction that writes one of them in the
two wait states behind it changes what is stored: in ``lora_add`` an offset came to lie in the place of two values of y.
The compiler keeps that distance, but not for buffer stores with an offset in a scalar register, so every kernel of the
built library is looked through, along both ways of each branch."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from block_wise_int8_amd import build

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WAIT_STATES = 2
WIDE = re.compile(r"(buffer|global|flat|scratch)_store_dwordx[34]")
LINE = re.compile(r"\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):")
TARGET = re.compile(r"<(.+?)(?:\+0x([0-9a-f]+))?>\s*$")


def registers(operand):
    """The vector registers of an operand, as (kind, number)."""
    m = re.match(r"([va])(?:(\d+)|\[(\d+):(\d+)\])$", operand)
    if not m:
        return set()
    first, last = (m[2], m[2]) if m[2] else (m[3], m[4])
    return {(m[1], n) for n in range(int(first), int(last) + 1)}


def parse(text):
    """[(mnemonic, operands, the branch's target or None)] in order, and the place of each address."""
    code, places, symbols = [], {}, {}
    for line in text.splitlines():
        head = re.match(r"([0-9a-f]{16}) <(.+)>:$", line)
        if head:
            symbols[head[2]] = int(head[1], 16)
            continue
        m = LINE.match(line)
        if m:
            places[int(m[3], 16)] = len(code)
            target = TARGET.search(line) if m[1].startswith(("s_branch", "s_cbranch")) else None
            code.append((m[1], [o.strip() for o in m[2].split(",")], target and (target[1], int(target[2] or "0", 16))))
    resolve = lambda t: None if t is None else places.get(symbols.get(t[0], -1) + t[1])
    return [(name, operands, resolve(t)) for name, operands, t in code]


def overwritten(code):
    """The stores of which a vector instruction within the wait states writes a register of the data."""
    found = []
    for i, (name, operands, _) in enumerate(code):
        if not WIDE.match(name):
            continue
        data = registers(operands[0] if name.startswith("buffer") else operands[1])
        assert len(data) in (3, 4), (name, operands)
        ways = [(i + 1, 0)]
        while ways:
            at, waited = ways.pop()
            if waited >= WAIT_STATES or at >= len(code):
                continue
            name2, operands2, target = code[at]
            if name2.startswith("v_") and data & registers(operands2[0]):
                found.append((name, operands, name2, operands2))
            if name2 == "s_endpgm":
                continue
            waited += int(operands2[0], 0) + 1 if name2 == "s_nop" else 1
            if target is not None:
                ways.append((target, waited))
            if name2 != "s_branch":
                ways.append((at + 1, waited))
    return found


def test_the_search():
    """A store whose data is overwritten at once, one instruction later and beyond a branch is found; later is not."""
    def listing(*lines):
        return parse("0000000000000100 <k>:\n" + "\n".join("\t%s // %012X: 00" % (l, 0x100 + 4 * i) + (
            " <k+0x10>" if l.startswith("s_branch") else "") for i, l in enumerate(lines)))

    store = "buffer_store_dwordx4 v[6:9], v22, s[12:15], s71 offen"
    assert len(overwritten(listing(store, "v_cndmask_b32_e64 v6, v67, v70, s[0:1]"))) == 1
    assert len(overwritten(listing(store, "s_nop 0", "v_mov_b32_e32 v9, 0"))) == 1
    assert len(overwritten(listing(store, "s_branch 2", "v_mov_b32_e32 v8, 0", "s_nop 0", "v_mov_b32_e32 v7, 0"))) == 1
    assert not overwritten(listing(store, "s_nop 1", "v_mov_b32_e32 v6, 0"))
    assert not overwritten(listing(store, "v_mov_b32_e32 v5, v6", "v_mov_b32_e32 v10, v9", "v_mov_b32_e32 v6, 0"))
    assert len(overwritten(listing("global_store_dwordx4 v[0:1], v[2:5], off", "v_mov_b32_e32 v5, 0"))) == 1
    assert not overwritten(listing("global_store_dwordx4 v[0:1], v[2:5], off", "v_mov_b32_e32 v1, 0"))


def test_no_wide_store_is_overwritten(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(build.LIB_PATH):
        build.build()
    shutil.copy(build.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    objects = glob.glob(str(tmp_path / ("lib.so.*" + build.ARCH)))
    assert objects
    stores = 0
    for path in objects:
        text = subprocess.run([OBJDUMP, "-d", path], check=True, capture_output=True, text=True).stdout
        code = parse(text)
        stores += sum(1 for name, _, _ in code if WIDE.match(name))
        assert overwritten(code) == []
    assert stores > 100   # (the listing was read)
