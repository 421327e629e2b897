"""Low-rank adapters again and again on the same inputs, alone and beside traffic that makes memory slow: every call
gives the bits of the first, which is held against the oracle (tolerance: see test_gpu_lora).  The order of the sums goes
by the sizes alone, so nothing may differ.  Sizes are those of whole and broken steps of columns, of rows that begin on
cache lines and beside them, of tiles of rows of each kind and of ranks that share registers in their own ways."""
import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import workloads as wl
from gpu_util import bf16_bits, bf16_to_dev, device, to_dev
from test_gpu_lora import check, make

pytestmark = pytest.mark.gpu

CALLS = 12


def runs(rng, M, L, n, bare):
    """Rows of n requests one behind the other, each with an adapter or none."""
    of = np.where(rng.random(n) < bare, -1, rng.integers(0, L, n))
    return of[np.sort(rng.integers(0, n, M))].astype(np.int32)


@pytest.mark.parametrize("M,N,K,L,R,parts,xpad,ypad,n", [
    (333, 5000, 4000, 5, 8, None, 96, 0, 40), (333, 5000, 4000, 5, 8, None, 96, 56, 40), (333, 5120, 4000, 5, 8, None, 96, 0, 40),
    (333, 4999, 515, 5, 8, None, 0, 0, 40), (64, 6144, 512, 64, 16, (4096, 1024, 1024), 0, 0, 64), (16, 4136, 256, 3, 24, None, 0, 0, 4),
    (500, 2600, 264, 4, 64, (1304, 1296), 0, 8, 9), (400, 2088, 264, 3, 96, None, 0, 0, 9), (300, 1064, 264, 3, 128, None, 0, 0, 5),
    (300, 1064, 264, 3, 256, None, 0, 0, 5), (700, 3000, 128, 2, 40, (1000, 2000), 8, 0, 60), (300, 1032, 264, 600, 32, None, 0, 0, 300)])
def test_every_call_gives_the_same_bits(M, N, K, L, R, parts, xpad, ypad, n):
    for seed in range(3):
        rng = wl.rng_for((141, seed, M, N, R, ypad))
        x, a, b, _, s = make(rng, M, N, K, L, R, 1 if parts is None else len(parts), pad=xpad)
        wide = wl.activations(rng, M, N + ypad)
        adapter = runs(rng, M, L, n, 0.2)
        args = [bf16_to_dev(x)[:, :K], bf16_to_dev(a), bf16_to_dev(b), to_dev(adapter), to_dev(s), parts]
        y = bf16_to_dev(wide)
        ys = [y.clone() for _ in range(CALLS)]
        traffic, other = torch.cuda.Stream(), torch.zeros(1 << 26, dtype=torch.float32, device=device())
        torch.cuda.synchronize()
        for i, out in enumerate(ys):
            if i % 2:   # the card's memory is busy with something else
                with torch.cuda.stream(traffic):
                    other.add_(1.0)
            bi8.lora_add(out[:, :N], *args)
        torch.cuda.synchronize()
        bits = [bf16_bits(t) for t in ys]
        for got in bits[1:]:
            differ = np.argwhere(got != bits[0])
            assert not len(differ), (seed, len(differ), [(r, c, adapter[r], hex(bits[0][r, c]), hex(got[r, c])) for r, c in differ[:8]])
        assert np.array_equal(bits[0][:, N:], wide[:, N:])
        check(np.ascontiguousarray(bits[0][:, :N]), x[:, :K], a, b, wide[:, :N], s, adapter, parts or (N,))
