"""One workspace, kept for the largest batch, serves the smaller ones: the same bits as with a fresh one."""
import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import workloads as wl
from gpu_util import bf16_to_dev, device, to_dev
from test_gpu_lora import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("largest,M", [(2049, 2048), (4097, 4096), (4097, 2048), (4097, 1)])
def test_adapters(largest, M):
    rng = wl.rng_for((151, M))
    N, K, L, R = 40, 4096, 3, 8
    x, a, b, y, s = [t if t.dtype == np.float32 else bf16_to_dev(t) for t in make(rng, M, N, K, L, R, 1)]
    args = [x, a, b, to_dev(rng.integers(-1, L, M).astype(np.int32)), to_dev(s)]
    scratch = torch.full((bi8.lora_add_workspace_size(largest, K, R),), 0xFF, dtype=torch.uint8, device=device())
    assert torch.equal(bi8.lora_add(y.clone(), *args, workspace=scratch), bi8.lora_add(y.clone(), *args))


@pytest.mark.parametrize("largest,T", [(4097, 4096), (8193, 8192), (16384, 4096), (16384, 100)])
def test_router(largest, T):
    logits = to_dev(wl.rng_for((152, T)).standard_normal((T, 24)).astype(np.float32))
    scratch = torch.full((bi8.moe_route_grouped_workspace_size(largest, 24),), 0xFF, dtype=torch.uint8, device=device())
    for one, other in zip(bi8.moe_route_grouped(logits, 3, workspace=scratch), bi8.moe_route_grouped(logits, 3)):
        assert torch.equal(one, other)
