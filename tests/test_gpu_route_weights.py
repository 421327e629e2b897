"""Weights of a softmax that is not renormalised: scores, sum and scale in binary64, rounded once, so within 2^-24 of
the oracle's (1.01 of it for the binary64 steps).  Rows of one large logit and many equal smaller ones, where an
exponential's error would not average out."""
import numpy as np
import pytest

import block_wise_int8_amd as bi8
import workloads as wl
from gpu_util import to_dev
from oracle import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,groups,scale", [
    (1, 64, 2, 1, 1.0), (40, 256, 8, 8, 1.0), (64, 1000, 4, 1, 2.5), (1500, 160, 6, 8, 16.0), (300, 512, 3, 4, 1.0),
    (20, 1023, 9, 33, 1.0)])
def test_rounded_once(T, E, k, groups, scale):
    rng = wl.rng_for((161, T, E))
    l = np.repeat(rng.uniform(-1, 1, (T, 1)), E, 1)
    l[np.arange(T), rng.integers(0, E, T)] += rng.uniform(0.5, 6, T)
    l = l.astype(np.float32)
    l[: T // 3] += (3 * rng.standard_normal((T // 3, E))).astype(np.float32)
    ids, w = [t.cpu().numpy() for t in bi8.moe_route_grouped(to_dev(l), k, groups=groups, topk_groups=max(1, groups // 2 + 1),
                                                             scale=scale)[:2]]
    want, wt = layer.route_grouped(l, k, "softmax", None, groups, max(1, groups // 2 + 1), 1, False, scale)
    assert np.array_equal(ids, want)
    assert np.all(np.abs(w - wt) <= 1.01 * 2.0 ** -24 * np.abs(wt))
