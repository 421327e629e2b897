"""The same 128 rotated values by each way through the kernel: the same bits.

The chunk that a lane holds goes by the head's size, the pairs and the pairing alone: 8 values where both halves of a
head are multiples of 8 (with nothing behind the rotation, and with), 4, 1, and several units a lane in long heads.  The
table is read four values at a time where axes and its address allow, else one at a time."""
import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import workloads as wl
from gpu_util import bf16_bits, bf16_to_dev, device, to_dev
from test_gpu_heads import gain, rope_table

pytestmark = pytest.mark.gpu

ROT, P = 128, 40


def tables():
    """The table at a 16-byte address and one value behind one."""
    table = rope_table(P, ROT)
    room = torch.zeros(P * ROT + 4, dtype=torch.float32, device=device())
    one = room[1: 1 + P * ROT].view(P, ROT)
    one.copy_(to_dev(table))
    assert to_dev(table).data_ptr() % 16 == 0 and one.data_ptr() % 16 == 4
    return to_dev(table), one


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (37, 3)])
def test_sizes_of_heads(T, H, interleaved):
    rng = wl.rng_for((171, T, H))
    x = wl.activations(rng, T, H * ROT).reshape(T, H, ROT)
    positions = rng.integers(0, P, T).astype(np.int32)
    want = None
    for D in (128, 136, 132, 130, 516, 640, 1022):
        wide = wl.activations(rng, T, H * D).reshape(T, H, D)
        wide[:, :, :ROT] = x
        for table in tables():
            for sections in ((64,), (32, 32), (33, 31), (1, 2, 61)):
                pos = to_dev(np.tile(positions, (len(sections), 1)))
                got = bf16_bits(bi8.qk_norm_rope(bf16_to_dev(wide), None, pos, table, sections=sections, interleaved=interleaved)[0])
                want = got if want is None else want
                assert np.array_equal(got[:, :, :ROT], want[:, :, :ROT]), (D, sections)
                assert np.array_equal(got[:, :, ROT:], wide[:, :, ROT:]), (D, sections)   # not turned: as they were


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H", [(1, 2), (900, 5)])
def test_the_tables_address_and_axes_beside_a_norm(T, H, interleaved):
    rng = wl.rng_for((172, T))
    x, w = bf16_to_dev(wl.activations(rng, T, H * ROT).reshape(T, H, ROT)), bf16_to_dev(gain(rng, ROT))
    positions = rng.integers(0, P, T).astype(np.int32)
    calls = [bi8.qk_norm_rope(x, None, to_dev(np.tile(positions, (len(s), 1))), t, w, sections=s, interleaved=interleaved)[0]
             for t in tables() for s in ((64,), (32, 32), (33, 31))]
    assert all(torch.equal(calls[0], got) for got in calls)
