"""Sizes of an MX4 product that no launch takes are refused before anything
is allocated or enqueued (on the CPU: nothing here reaches a device)."""
import pytest

import dense_tiled_gemm_fp16_amd as g

P = [0x100000000000 + (i << 43) for i in range(5)]   # never dereferenced
SHAPE = -2


@pytest.mark.parametrize("M,N", [(1 << 20, 1 << 20), (1 << 31, 129), (129, 1 << 31), (1 << 25, 1 << 15)])
@pytest.mark.parametrize("workspace", [None, 0x700000000000])
def test_more_tiles_than_a_launch_takes(M, N, workspace):
    K = 32
    need = g.gemm_mx4_workspace_bytes(M, N, K)
    assert need > 0
    rc = g.lib.gemm_mx4(P[0], 16, P[1], 1, P[2], 16, P[3], 1, P[4], 0, N, M, N, K, None, workspace, need)
    assert rc == SHAPE
