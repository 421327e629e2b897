"""Workspaces of the operators beside the 8-bit products: a size does not fall as batches grow, so that a program that
keeps one for its largest batch has enough for each."""
import pytest

import block_wise_int8_amd as bi8


@pytest.mark.parametrize("K,R,parts", [(4096, 64, 1), (4096, 16, 3), (1100, 24, 2), (64, 8, 1), (9000, 256, 1), (600, 128, 2)])
def test_adapters(K, R, parts):
    sizes = [bi8.lora_add_workspace_size(M, K, R, parts) for M in range(1, 17000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert all(n >= M * R * parts * 4 for M, n in enumerate(sizes, 1))
    # from where a row needs one sum: nothing more than that
    assert bi8.lora_add_workspace_size(1 << 20, K, R, parts) == (1 << 20) * R * parts * 4


@pytest.mark.parametrize("E", [1, 8, 160, 256, 1021])
def test_router(E):
    sizes = [bi8.moe_route_grouped_workspace_size(T, E) for T in range(1, 18000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
