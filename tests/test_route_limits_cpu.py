"""The router's largest batch (no GPU, no kernel launched): more tokens than its launches hold threads for are refused as
a size, before any HIP call."""
import pytest

import block_wise_int8_amd as bi8

P, SHAPE = 0x10000, 2
MOST = (1 << 28) - 64


@pytest.mark.parametrize("T,k", [(MOST + 1, 1), (1 << 28, 7), ((1 << 31) - 1, 1), (MOST, 9), (1 << 27, 16)])
def test_too_many_tokens(T, k):
    lib = bi8.load()
    status = lib.blockint8_moe_route_grouped(P, 0, 64, None, T, 64, k, 0, 1, 1, 1, 0, 1.0, P, P, P, P, P, P, 1 << 60, None)
    assert status == SHAPE and b"T = %d out of range" % T in lib.blockint8_last_error()


def test_the_most_tokens():
    """Their workspace is of a size, and asked for: the next check."""
    lib = bi8.load()
    assert bi8.moe_route_grouped_workspace_size(MOST, 64) > 0 == bi8.moe_route_grouped_workspace_size(MOST + 1, 64)
    status = lib.blockint8_moe_route_grouped(P, 0, 64, None, MOST, 64, 7, 0, 1, 1, 1, 0, 1.0, P, P, P, P, P, P, 16, None)
    assert status == SHAPE and b"workspace_bytes" in lib.blockint8_last_error()
